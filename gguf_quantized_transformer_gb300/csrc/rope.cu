// Rotary positions as a standalone operator: pairs (a, b) of a head's first R dims are rotated by
// theta = pos * f_i and scaled by a magnitude m,
//   y_a = m (x_a cos theta - x_b sin theta),   y_b = m (x_a sin theta + x_b cos theta),
// with (a, b) = (2i, 2i + 1) (interleaved) or (i, i + R/2) (half); the other dims are copied.
//
// The angle: f_i / 2 pi is a 64-bit fixed-point fraction of a turn computed on the host in fp64, and pos times it
// modulo 2^64 is the angle modulo a turn.  What fp64 rounds off f_i / 2 pi (a power built by repeated products: at
// most 2^-53 of a turn, since i base^(-2i / R) / 2 pi stays below 1) grows with pos: 2^-33 of a turn at a million
// positions, 2^-22 at 2^31.  The integer is reduced to the nearest quarter turn before it becomes a float, so the
// argument of sin and cos is off by at most 2^-24 of its own value, itself at most pi / 4.
//
// Bound by HBM: every value is read and written once.  A thread owns a vector of pairs of one row and computes its
// sines once for the heads it walks.
#include "draft.cuh"

namespace af {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void turn_sincos(uint64_t turn, int pos, float mag, float& c, float& s) {
    const uint64_t t = (uint64_t)((int64_t)pos) * turn;            // modulo one turn
    const unsigned quad = (unsigned)((t + (1ull << 61)) >> 62);     // nearest quarter turn
    const int rem = (int)((int64_t)(t << 2) >> 32);                 // the rest: [-1/8, 1/8) turn in 2^-34 turns
    float sn, cs;
    sincospif((float)rem * 0x1p-33f, &sn, &cs);
    const float c0 = (quad & 1) ? -sn : cs, s0 = (quad & 1) ? cs : sn;
    c = mag * ((quad & 2) ? -c0 : c0);
    s = mag * ((quad & 2) ? -s0 : s0);
}

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T e[N];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __half& o) { o = __float2half_rn(v); }

// V consecutive elements per access.  A unit of a head is: half layout, V pairs (elements i..i+V-1 and the same
// + R/2); interleaved, V / 2 pairs (V consecutive elements; V = 1: one pair, two accesses of one element); past R,
// V copied elements.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const T* x, T* y, int64_t ldx, int64_t ldy, int n, int heads, int D, int R, const int* __restrict__ pos,
                int pos0, float mag, int hgroups, const __grid_constant__ RopeTurns turns) {
    constexpr int P = HALF ? V : (V > 1 ? V / 2 : 1);  // pairs per unit
    const int rot_units = R / 2 / P, copy_units = (D - R) / V, units = rot_units + copy_units;
    const int64_t total = (int64_t)n * hgroups * units;
    for (int64_t w = (int64_t)blockIdx.x * kThreads + threadIdx.x; w < total; w += (int64_t)gridDim.x * kThreads) {
        const int u = (int)(w % units);
        const int64_t rg = w / units;
        const int hg = (int)(rg % hgroups);
        const int64_t row = rg / hgroups;
        const T* xr = x + row * ldx;
        T* yr = y + row * ldy;
        if (u >= rot_units) {
            const int d = R + (u - rot_units) * V;
            for (int h = hg; h < heads; h += hgroups)
                *reinterpret_cast<Vec<T, V>*>(yr + h * D + d) = *reinterpret_cast<const Vec<T, V>*>(xr + h * D + d);
            continue;
        }
        const int p = pos ? pos[row] : pos0 + (int)row;
        float c[P], s[P];
#pragma unroll
        for (int e = 0; e < P; e++) turn_sincos(turns.turn[u * P + e], p, mag, c[e], s[e]);
        for (int h = hg; h < heads; h += hgroups) {
            if (HALF) {
                const int64_t ia = (int64_t)h * D + u * V, ib = ia + R / 2;
                const Vec<T, V> a = *reinterpret_cast<const Vec<T, V>*>(xr + ia);
                const Vec<T, V> b = *reinterpret_cast<const Vec<T, V>*>(xr + ib);
                Vec<T, V> oa, ob;
#pragma unroll
                for (int e = 0; e < V; e++) {
                    const float fa = to_f(a.e[e]), fb = to_f(b.e[e]);
                    from_f(fa * c[e] - fb * s[e], oa.e[e]);
                    from_f(fa * s[e] + fb * c[e], ob.e[e]);
                }
                *reinterpret_cast<Vec<T, V>*>(yr + ia) = oa;
                *reinterpret_cast<Vec<T, V>*>(yr + ib) = ob;
            } else {
                constexpr int W = V > 1 ? V : 2;
                constexpr int A = V > 1 ? V : 1;  // elements per access
                const int64_t i0 = (int64_t)h * D + u * W;
                alignas(16) T in[W], out[W];
#pragma unroll
                for (int e = 0; e < W; e += A) *reinterpret_cast<Vec<T, A>*>(in + e) = *reinterpret_cast<const Vec<T, A>*>(xr + i0 + e);
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                    const float fa = to_f(in[e]), fb = to_f(in[e + 1]);
                    from_f(fa * c[e / 2] - fb * s[e / 2], out[e]);
                    from_f(fa * s[e / 2] + fb * c[e / 2], out[e + 1]);
                }
#pragma unroll
                for (int e = 0; e < W; e += A) *reinterpret_cast<Vec<T, A>*>(yr + i0 + e) = *reinterpret_cast<const Vec<T, A>*>(out + e);
            }
        }
    }
}

template <typename T, int V, bool HALF>
cudaError_t go(const RopeArgs& a, const RopeTurns& t, cudaStream_t s) {
    constexpr int P = HALF ? V : (V > 1 ? V / 2 : 1);
    const int64_t units = a.R / 2 / P + (a.D - a.R) / V;
    const int64_t room = (int64_t)num_sms() * 2048;
    int64_t hg = (room + a.n * units - 1) / (a.n * units);  // head groups: enough threads to fill the card
    if (hg > a.heads) hg = a.heads;
    if (hg < 1) hg = 1;
    int64_t blocks = (a.n * hg * units + kThreads - 1) / kThreads;
    if (blocks > (int64_t)num_sms() * 64) blocks = (int64_t)num_sms() * 64;
    rope_kernel<T, V, HALF><<<(unsigned)blocks, kThreads, 0, s>>>((const T*)a.x, (T*)a.y, a.ldx, a.ldy, a.n, a.heads, a.D,
                                                                   a.R, a.pos, a.pos0, a.mag, (int)hg, t);
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const RopeArgs& a, const RopeTurns& t, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    // 16-byte accesses where every vector of every row starts on 16 bytes and none crosses the rotated part's end
    const bool al = (((uintptr_t)a.x | (uintptr_t)a.y) & 15) == 0 && a.ldx % V == 0 && a.ldy % V == 0 && a.D % V == 0 &&
                    (a.half ? a.R / 2 : a.R) % V == 0;
    if (a.half) return al ? go<T, V, true>(a, t, s) : go<T, 1, true>(a, t, s);
    return al ? go<T, V, false>(a, t, s) : go<T, 1, false>(a, t, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, const RopeTurns& t, cudaStream_t s) {
    return a.f16 ? pick<__half>(a, t, s) : pick<float>(a, t, s);
}

}  // namespace af

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
// Sine and cosine on [-pi / 4, pi / 4] are their Taylor series (remainders below 2^-28 and 2^-33), two pairs at a time
// in packed fp32.
//
// Every value is read and written once.  A thread keeps one unit of the head (its frequencies in registers) and walks rows
// with it, and the heads of a row with the sines of that row.  4096 rows x 40 x 128: fp32 32.8 us (half) and 36.2
// (interleaved), fp16 26.3 and 20.9; 245760 rows x 128 of one position: 45.5, 49.4, 34.5 and 37.7: 3.2 to 5.5 TB/s, bound
// by each thread's wait for its own loads (16 to 24 warps an SM).
#include "draft.cuh"
#include "tma.cuh"

namespace af {

namespace {

constexpr int kThreads = 256;

// mag cos and mag sin of pos * turn, for two frequencies
__device__ __forceinline__ void turn_sincos2(const uint64_t (&turn)[2], int pos, float mag, float2& co, float2& so) {
    unsigned quad[2];
    float x[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint64_t t = (uint64_t)((int64_t)pos) * turn[i];     // modulo one turn
        const unsigned h = (unsigned)(t >> 32);                     // (what lies below is 2^-32 of a turn)
        quad[i] = (h + (1u << 29)) >> 30;                           // nearest quarter turn
        x[i] = (float)(int)((unsigned)(t >> 30));                   // the rest in 2^-34 turns, [-1/8, 1/8) turn
    }
    const float2 a = mul2(make_float2(x[0], x[1]), both(3.14159265358979f * 0x1p-33f)), z = mul2(a, a);
    float2 sn = fma2(z, both(1.f / 362880), both(-1.f / 5040));
    sn = fma2(z, sn, both(1.f / 120));
    sn = fma2(z, sn, both(-1.f / 6));
    sn = fma2(mul2(z, a), sn, a);
    float2 cs = fma2(z, both(-1.f / 3628800), both(1.f / 40320));
    cs = fma2(z, cs, both(-1.f / 720));
    cs = fma2(z, cs, both(1.f / 24));
    cs = fma2(z, cs, both(-0.5f));
    cs = fma2(z, cs, both(1.f));
    const float2 m = both(mag);
    sn = mul2(sn, m);
    cs = mul2(cs, m);
    const float sv[2] = {sn.x, sn.y}, cv[2] = {cs.x, cs.y};
    float c[2], s[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {  // quarter turns: (c, s) -> (-s, c)
        const float c0 = (quad[i] & 1) ? -sv[i] : cv[i], s0 = (quad[i] & 1) ? cv[i] : sv[i];
        const unsigned flip = (quad[i] & 2) << 30;
        c[i] = __uint_as_float(__float_as_uint(c0) ^ flip);
        s[i] = __uint_as_float(__float_as_uint(s0) ^ flip);
    }
    co = make_float2(c[0], c[1]);
    so = make_float2(s[0], s[1]);
}

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T e[N];
};
// N values through L2 (an earlier kernel of the chain may have written them)
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load(const T* p) {
    Vec<T, N> v;
    if constexpr (sizeof(T) * N == 16)
        *reinterpret_cast<uint4*>(&v) = __ldcg(reinterpret_cast<const uint4*>(p));
    else if constexpr (sizeof(T) * N == 4)
        *reinterpret_cast<unsigned*>(&v) = __ldcg(reinterpret_cast<const unsigned*>(p));
    else
        *reinterpret_cast<unsigned short*>(&v) = __ldcg(reinterpret_cast<const unsigned short*>(p));
    return v;
}

// values e and e + 1 of a vector, as fp32 and back
template <int N>
__device__ __forceinline__ float2 pair_of(const Vec<float, N>& v, int e) { return make_float2(v.e[e], v.e[e + 1]); }
template <int N>
__device__ __forceinline__ float2 pair_of(const Vec<__half, N>& v, int e) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v.e[e]));
}
template <int N>
__device__ __forceinline__ void set_pair(Vec<float, N>& v, int e, float2 x) { v.e[e] = x.x, v.e[e + 1] = x.y; }
template <int N>
__device__ __forceinline__ void set_pair(Vec<__half, N>& v, int e, float2 x) {
    *reinterpret_cast<__half2*>(&v.e[e]) = __floats2half2_rn(x.x, x.y);
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __half& o) { o = __float2half_rn(v); }

// A unit of a head is, in accesses of V values: half layout, V pairs (elements i..i+V-1 and the same + R/2);
// interleaved, V / 2 pairs (V consecutive elements; V = 1: one pair, two accesses); past R, V copied elements.
// Rows are n * hgroups: (row, heads hg, hg + hgroups, ..).
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads, HALF && V > 4 ? 2 : 3)
    rope_kernel(const T* x, T* y, int64_t ldx, int64_t ldy, int n, int heads, int D, int R, const int* __restrict__ pos,
                int pos0, float mag, int hgroups, int units, int rows_per_cta, const __grid_constant__ RopeTurns turns) {
    constexpr int P = HALF ? V : (V > 1 ? V / 2 : 1), P2 = P > 1 ? P : 2;  // pairs per unit
    const int rot_units = R / 2 / P;
    // the rotating threads of all the CTA's rows come first: few warps hold both kinds
    const int tid = threadIdx.x, nrot = rot_units * rows_per_cta;
    const bool copy = tid >= nrot;
    const int rl = copy ? (tid - nrot) / max(units - rot_units, 1) : tid / rot_units;
    const int u = copy ? rot_units + (tid - nrot) % max(units - rot_units, 1) : tid % rot_units;
    // (through shared memory: lanes that read parameters at different offsets take turns)
    __shared__ uint64_t turn[kRopeMaxPairs];
    if (tid < R / 2) turn[tid] = turns.turn[tid];
    __syncthreads();
    uint64_t tn[P2];
#pragma unroll
    for (int e = 0; e < P2; e++) tn[e] = !copy && e < P ? turn[u * P + e] : 0;
    pdl_wait();
    // The accesses of this thread's unit in a head: NA of A values.
    constexpr int W = HALF ? V : (V > 1 ? V : 2), A = HALF ? V : (V > 1 ? V : 1), NA = HALF ? 2 : W / A;
    const int first = copy ? R + (u - rot_units) * V : u * W, step = HALF ? R / 2 : A;
    struct Unit {
        Vec<T, A> v[NA];
    };
    auto get = [&](const T* p) {
        Unit x;
        x.v[0] = load<T, A>(p + first);
#pragma unroll
        for (int e = 1; e < NA; e++)
            if (!copy) x.v[e] = load<T, A>(p + first + e * step);
        return x;
    };
    auto put = [&](T* p, Unit x, const float2 (&c)[P2 / 2], const float2 (&s)[P2 / 2]) {
        if (!copy) {
            if constexpr (V == 1) {  // one pair in two accesses
                const float a = to_f(x.v[0].e[0]), b = to_f(x.v[1].e[0]);
                from_f(a * c[0].x - b * s[0].x, x.v[0].e[0]);
                from_f(a * s[0].x + b * c[0].x, x.v[1].e[0]);
            } else if constexpr (HALF) {
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float2 a = pair_of(x.v[0], e), b = pair_of(x.v[1], e), cc = c[e / 2], ss = s[e / 2];
                    set_pair(x.v[0], e, fma2(mul2(b, ss), both(-1.f), mul2(a, cc)));
                    set_pair(x.v[1], e, fma2(a, ss, mul2(b, cc)));
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; e += 2) {  // pair e / 2
                    const float2 ab = pair_of(x.v[0], e);
                    const float ce = e & 2 ? c[e / 4].y : c[e / 4].x, se = e & 2 ? s[e / 4].y : s[e / 4].x;
                    set_pair(x.v[0], e, fma2(make_float2(-ab.y, ab.x), both(se), mul2(ab, both(ce))));
                }
            }
        }
        *reinterpret_cast<Vec<T, A>*>(p + first) = x.v[0];
#pragma unroll
        for (int e = 1; e < NA; e++)
            if (!copy) *reinterpret_cast<Vec<T, A>*>(p + first + e * step) = x.v[e];
    };
    if (tid >= units * rows_per_cta) return;
    const int64_t total = (int64_t)n * hgroups, stride = (int64_t)gridDim.x * rows_per_cta;
    // item w: row w / hgroups, first head w % hgroups (several head groups: total is a small number)
    auto row_of = [&](int64_t w) { return hgroups == 1 ? w : (int64_t)((unsigned)w / (unsigned)hgroups); };
    auto head_of = [&](int64_t w) { return hgroups == 1 ? 0 : (int)((unsigned)w % (unsigned)hgroups); };
    int64_t w = (int64_t)blockIdx.x * rows_per_cta + rl;
    if (w >= total) return;
    int64_t row = row_of(w);
    int hg = head_of(w);
    const T* xr = x + row * ldx;
    Unit cur = get(xr + hg * D);
    int p = pos ? __ldcg(pos + row) : pos0 + (int)row;
    float2 c[P2 / 2], s[P2 / 2];
    int p_of = 0;
    bool fresh = true;
    while (true) {
        // the next item's first head and position are on their way while this one is worked on
        const int64_t wn = w + stride;
        int64_t rn = row;
        int hn = hg, pn = 0;
        const T* xn = xr;
        Unit next = cur;
        if (wn < total) {
            rn = row_of(wn);
            hn = head_of(wn);
            xn = x + rn * ldx;
            next = get(xn + hn * D);
            pn = pos ? __ldcg(pos + rn) : pos0 + (int)rn;
        }
        T* yr = y + row * ldy;
        if (fresh || p != p_of) {  // rows that share a position (a cache that moves) share its sines
#pragma unroll
            for (int e = 0; e < P2; e += 2) {
                const uint64_t t2[2] = {tn[e], tn[e + 1]};
                turn_sincos2(t2, p, mag, c[e / 2], s[e / 2]);
            }
            p_of = p;
            fresh = false;
        }
        put(yr + hg * D, cur, c, s);
        for (int h = hg + hgroups; h < heads; h += 2 * hgroups) {
            const bool two = h + hgroups < heads;
            const Unit a = get(xr + h * D);
            Unit b = a;
            if (two) b = get(xr + (h + hgroups) * D);
            put(yr + h * D, a, c, s);
            if (two) put(yr + (h + hgroups) * D, b, c, s);
        }
        if (wn >= total) break;
        w = wn, row = rn, hg = hn, xr = xn, cur = next, p = pn;
    }
    __threadfence();  // (and no early launch of the next kernel: see launch_chained)
}

template <typename T, int V, bool HALF>
cudaError_t go(const RopeArgs& a, const RopeTurns& t, cudaStream_t s) {
    constexpr int P = HALF ? V : (V > 1 ? V / 2 : 1);
    const int units = a.R / 2 / P + (a.D - a.R) / V, rows = kThreads / units;  // (units <= 255: R >= 2, D <= 256)
    const int64_t room = (int64_t)num_sms() * 2048;
    int64_t hg = (room + a.n * (int64_t)units - 1) / (a.n * (int64_t)units);  // head groups: enough threads to fill the card
    hg = hg > a.heads ? a.heads : (hg < 1 ? 1 : hg);
    int64_t blocks = (a.n * hg + rows - 1) / rows;
    if (blocks > (int64_t)num_sms() * 8) blocks = (int64_t)num_sms() * 8;
    return launch_chained(rope_kernel<T, V, HALF>, dim3((unsigned)blocks), kThreads, 0, s, (const T*)a.x, (T*)a.y, a.ldx, a.ldy,
                          a.n, a.heads, a.D, a.R, a.pos, a.pos0, a.mag, (int)hg, units, rows, t);
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

// Writing rows of keys and values into a cache of any type, and reading slots back as fp32 rows.
//
// A quantized cache holds, per 32 values along head_dim, an fp16 scale d and integer codes q, value d q:
//   Q8_0: d = fp16(max|v| / 127), q = clamp(round-half-away(v / d), -127, 127)
//   Q4_0: d = fp16(m / -8) with m the value of largest magnitude (the first on ties),
//         q = clamp(floor(v / d + 1/2), -8, 7)
// with the decisions those of exact arithmetic: q is guessed as v times a 1 / d that is a little small, rounded, so it is
// right or one too near zero.  q d has at most 8 + 11 bits and is an fp32 number, and |q| d <= |v| < 2 |q| d (or q = 0),
// so r = v - q d comes out of one fused multiply-add exactly, and comparing r with d / 2 corrects the guess.  A zero d
// gives zero codes.  A block that holds a NaN, or whose scale overflows fp16, gets a NaN as its scale: nothing
// non-finite is turned into a number.
//
// A CTA takes a few rows at a time, all loads before the first use (writing: a thread holds eight values of a block, two
// float4 64 bytes apart, so that four lanes share a block's scale); the grid is a few CTAs per SM.  Data of earlier kernels
// is read through L2 (the kernels are launched with programmatic serialization).
// 30720 rows of 8 x 128, written and read: fp32 81 and 76 us, fp16 58 and 62, Q8_0 71 and 55, Q4_0 92 and 51, that is 5.7
// to 6.6 TB/s but for the quantizers' 4.5 and 3.1: those are bound by their instructions (issue slots 72% busy).
#include <algorithm>
#include <type_traits>

#include "draft.cuh"
#include "tma.cuh"

namespace af {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4, kWriteRows = 2, kGroup = 16;
constexpr int kCtasPerSm = 8;

// OR over the CTA, in every thread
__device__ __forceinline__ unsigned cta_or(unsigned x) {
    __shared__ unsigned part[kThreads / 32];
    x = __reduce_or_sync(0xffffffffu, x);
    __syncthreads();  // (the previous result has been read)
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) x |= part[w];
    return x;
}

// Four lanes (an aligned group of the warp) hold the 32 values of a block: lane i of them quads i and 4 + i.  Every lane of
// the warp takes part in the exchanges (with a mask per group the warp would run group by group: a quarter
// longer for 30720 rows of 8 x 128 values into Q4_0).
template <int TYPE>
__device__ __forceinline__ void quantize_group(const float (&x)[8], int lane, int (&q)[8], __half& dh) {
    unsigned amax = 0;  // magnitudes order like their bits, NaNs above infinity
#pragma unroll
    for (int e = 0; e < 8; e++) amax = max(amax, __float_as_uint(x[e]) & 0x7FFFFFFFu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    float m = __uint_as_float(amax);
    if (TYPE == AF_KV_Q8_0) {
        m = m / 127.f;
    } else {
        // the sign of the first value of that magnitude: of the first quads (by lane), then of the second
        unsigned mine = 0;  // 1: in the first quad, 2: in the second; << 2: negative there
#pragma unroll
        for (int e = 7; e >= 0; e--)
            if ((__float_as_uint(x[e]) & 0x7FFFFFFFu) == amax) {
                const unsigned w = e < 4 ? 1u : 2u;
                mine = (mine & ~(w << 2)) | w | (__float_as_uint(x[e]) >> 31 ? w << 2 : 0u);
            }
        const unsigned group = 0xfu << (lane & 28);
        const unsigned first = __ballot_sync(0xffffffffu, mine & 1) & group;
        const unsigned second = __ballot_sync(0xffffffffu, mine & 2) & group;
        const int src = first ? __ffs(first) - 1 : second ? __ffs(second) - 1 : lane;
        const unsigned theirs = __shfl_sync(0xffffffffu, mine, src);
        const bool negative = theirs & (first ? 4u : 8u);
        m = negative ? m * 0.125f : m * -0.125f;
    }
    dh = __float2half_rn(m);
    if ((__half_as_ushort(dh) & 0x7C00) == 0x7C00) dh = __ushort_as_half((unsigned short)0x7FFF);
    const float d = fabsf(__half2float(dh)), h = 0.5f * d;
    float rd;
    asm("rcp.approx.f32 %0, %1;" : "=f"(rd) : "f"(d));
    rd *= 1.f - 0x1p-20f;  // (the approximation is off by 2^-23)
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, in the low bits
#pragma unroll
    for (int e = 0; e < 8; e++) {
        // the rounding is half away from zero on |v| for Q8_0, half up on v / d for Q4_0: half up on y / |d| either way
        const float y = TYPE == AF_KV_Q8_0 ? fabsf(x[e]) : (__half_as_ushort(dh) & 0x8000 ? -x[e] : x[e]);
        const float g = fmaf(y, rd, kMagic);
        const float r = fmaf(-(g - kMagic), d, y);
        int v = __float_as_int(g) - 0x4B400000;
        v += (r >= h ? 1 : 0) - (r < -h ? 1 : 0);
        v = TYPE == AF_KV_Q8_0 ? min(v, 127) : min(max(v, -8), 7);
        if (TYPE == AF_KV_Q8_0 && x[e] < 0.f) v = -v;
        q[e] = d > 0.f ? v : 0;
    }
}

// The thread's eight values (at dims d0.. and d0 + 16.. of cell `cell`) into the cache.
template <int TYPE>
__device__ __forceinline__ void store_group(void* base, __half* scales, int64_t cell, int D, int d0, const float (&x)[8],
                                            int lane, bool in) {
    int q[8];
    __half dh;
    if (TYPE == AF_KV_Q8_0 || TYPE == AF_KV_Q4_0) quantize_group<TYPE>(x, lane, q, dh);
    if (!in) return;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        const int d = d0 + 4 * e;
        if (TYPE == AF_F32) {
            *reinterpret_cast<float4*>((float*)base + cell * D + d) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        } else if (TYPE == AF_F16) {
            __half2 h[2] = {__floats2half2_rn(x[e], x[e + 1]), __floats2half2_rn(x[e + 2], x[e + 3])};
            *reinterpret_cast<uint2*>((__half*)base + cell * D + d) = *reinterpret_cast<const uint2*>(h);
        } else if (TYPE == AF_KV_Q8_0) {
            *reinterpret_cast<unsigned*>((uint8_t*)base + cell * D + d) =
                __byte_perm(__byte_perm(q[e], q[e + 1], 0x0040), __byte_perm(q[e + 2], q[e + 3], 0x0040), 0x5410);
        } else {
            *reinterpret_cast<unsigned short*>((uint8_t*)base + cell * (D / 2) + d / 2) =
                (unsigned short)((q[e] + 8) | (q[e + 1] + 8) << 4 | (q[e + 2] + 8) << 8 | (q[e + 3] + 8) << 12);
        }
    }
    if ((TYPE == AF_KV_Q8_0 || TYPE == AF_KV_Q4_0) && (lane & 3) == 0) scales[cell * (D / 32) + d0 / 32] = dh;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(KvRows c, const float* __restrict__ k, const float* __restrict__ v, int64_t ld, int n,
                    const int* __restrict__ slots, int slot0, int group) {
    const int lane = threadIdx.x & 31;
    const int octs = c.KVH * c.D / 8;  // a multiple of 4
    pdl_wait();  // (and no early launch of the next kernel: see launch_chained)
    for (int g0 = blockIdx.x * group; g0 < n; g0 += gridDim.x * group) {
        unsigned again = 0;  // rows of the group whose slot a later row names too: it belongs to that one
        if (slots) {
            auto search = [&](auto rows) {
                constexpr int N = decltype(rows)::value;
                int named[N];
#pragma unroll
                for (int j = 0; j < N; j++) named[j] = j < group && g0 + j < n ? __ldcg(slots + g0 + j) : -1;
                for (int i = g0 + 1 + threadIdx.x; i < n; i += kThreads) {
                    const int x = __ldcg(slots + i);
#pragma unroll
                    for (int j = 0; j < N; j++) again |= (i > g0 + j && x == named[j]) ? 1u << j : 0u;
                }
            };
            if (group == kWriteRows)
                search(std::integral_constant<int, kWriteRows>());
            else
                search(std::integral_constant<int, kGroup>());
            again = cta_or(again);
        }
        for (int r0 = g0; r0 < min(n, g0 + group); r0 += kWriteRows, again >>= kWriteRows) {
            int slot[kWriteRows];  // -1: not written; the same in every thread of the CTA
#pragma unroll
            for (int j = 0; j < kWriteRows; j++) {
                slot[j] = r0 + j >= n ? -1 : slots ? __ldcg(slots + r0 + j) : slot0 + r0 + j;
                if (slot[j] >= c.ctx || (again >> j & 1)) slot[j] = -1;
            }
            for (int i0 = threadIdx.x - lane; i0 < 2 * octs; i0 += kThreads) {  // K, then V; whole warps
                const bool in = i0 + lane < 2 * octs;
                const int i = in ? i0 + lane : 0;
                const bool isv = i >= octs;
                const int b = (isv ? i - octs : i) >> 2, e0 = b * 32 + (i & 3) * 4, g = e0 / c.D, d0 = e0 - g * c.D;
                const float* src = (isv ? v : k) + r0 * ld + e0;
                float4 x[kWriteRows][2];
#pragma unroll
                for (int j = 0; j < kWriteRows; j++)
                    if (slot[j] >= 0) {
                        x[j][0] = __ldcg(reinterpret_cast<const float4*>(src + j * ld));
                        x[j][1] = __ldcg(reinterpret_cast<const float4*>(src + j * ld + 16));
                    }
#pragma unroll
                for (int j = 0; j < kWriteRows; j++)
                    if (slot[j] >= 0) {
                        const float a[8] = {x[j][0].x, x[j][0].y, x[j][0].z, x[j][0].w, x[j][1].x, x[j][1].y, x[j][1].z, x[j][1].w};
                        store_group<TYPE>(isv ? c.v : c.k, isv ? c.vs : c.ks, (int64_t)g * c.ctx + slot[j], c.D, d0, a, lane, in);
                    }
            }
        }
    }
    __threadfence();
}

// Four values as they lie in the cache, and as fp32.
template <int TYPE>
struct Cell4 {
    uint4 w;
    __half d;
};
template <int TYPE>
__device__ __forceinline__ void fetch4(const void* base, const __half* scales, int64_t cell, int D, int d0, Cell4<TYPE>& x) {
    if (TYPE == AF_F32) {
        x.w = __ldcg(reinterpret_cast<const uint4*>((const float*)base + cell * D + d0));
    } else if (TYPE == AF_F16) {
        const uint2 r = __ldcg(reinterpret_cast<const uint2*>((const __half*)base + cell * D + d0));
        x.w.x = r.x, x.w.y = r.y;
    } else {
        x.d = __ushort_as_half(__ldcg(reinterpret_cast<const unsigned short*>(scales) + cell * (D / 32) + d0 / 32));
        if (TYPE == AF_KV_Q8_0)
            x.w.x = __ldcg(reinterpret_cast<const unsigned*>((const uint8_t*)base + cell * D + d0));
        else
            x.w.x = __ldcg(reinterpret_cast<const unsigned short*>((const uint8_t*)base + cell * (D / 2) + d0 / 2));
    }
}
template <int TYPE>
__device__ __forceinline__ float4 value4(const Cell4<TYPE>& x) {
    if (TYPE == AF_F32) return *reinterpret_cast<const float4*>(&x.w);
    if (TYPE == AF_F16) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x.w.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&x.w.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    const float d = __half2float(x.d);
    const unsigned w = x.w.x;
    if (TYPE == AF_KV_Q8_0)
        return make_float4(d * (int8_t)(w & 255), d * (int8_t)(w >> 8 & 255), d * (int8_t)(w >> 16 & 255), d * (int8_t)(w >> 24));
    return make_float4(d * ((int)(w & 15) - 8), d * ((int)(w >> 4 & 15) - 8), d * ((int)(w >> 8 & 15) - 8),
                       d * ((int)(w >> 12) - 8));
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(KvRows c, int n, const int* __restrict__ slots, int slot0, float* __restrict__ k,
                   float* __restrict__ v, int64_t ld) {
    const int quads = c.KVH * c.D / 4;
    pdl_wait();  // (and no early launch of the next kernel: rows of one kv head are an fp32 cache, see launch_chained)
    for (int r0 = blockIdx.x * kRows; r0 < n; r0 += gridDim.x * kRows) {
        int slot[kRows];
#pragma unroll
        for (int j = 0; j < kRows; j++) {
            slot[j] = r0 + j >= n ? -1 : slots ? __ldcg(slots + r0 + j) : slot0 + r0 + j;
            if (slot[j] >= c.ctx) slot[j] = -1;
        }
        for (int i = threadIdx.x; i < quads; i += kThreads) {
            const int e0 = i * 4, g = e0 / c.D, d0 = e0 % c.D;
            Cell4<TYPE> x[2][kRows];
#pragma unroll
            for (int j = 0; j < kRows; j++)
                if (slot[j] >= 0) {
                    fetch4<TYPE>(c.k, c.ks, (int64_t)g * c.ctx + slot[j], c.D, d0, x[0][j]);
                    fetch4<TYPE>(c.v, c.vs, (int64_t)g * c.ctx + slot[j], c.D, d0, x[1][j]);
                }
#pragma unroll
            for (int j = 0; j < kRows; j++)
                if (slot[j] >= 0) {
                    *reinterpret_cast<float4*>(k + (r0 + j) * ld + e0) = value4<TYPE>(x[0][j]);
                    *reinterpret_cast<float4*>(v + (r0 + j) * ld + e0) = value4<TYPE>(x[1][j]);
                }
        }
    }
    __threadfence();
}

unsigned ctas(int n, int rows) { return (unsigned)std::min((n + rows - 1) / rows, num_sms() * kCtasPerSm); }

}  // namespace

cudaError_t launch_kv_write(const KvRows& c, const float* k, const float* v, int64_t ld, int n, const int* slots,
                            int slot0, cudaStream_t s) {
    // Rows that share one search for later rows of their slots: more where a CTA has more rows (30000 listed fp16 rows:
    // 203 us, 392 with searches for two rows; a run of slots 118)
    int group = kWriteRows;
    while (slots && group < kGroup && (int64_t)group * num_sms() * kCtasPerSm < n) group *= 2;
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3(ctas(n, group)), kThreads, 0, s, c, k, v, ld, n, slots, slot0, group);
    };
    switch (c.type) {
        case AF_F32: return go(kv_write_kernel<AF_F32>);
        case AF_F16: return go(kv_write_kernel<AF_F16>);
        case AF_KV_Q8_0: return go(kv_write_kernel<AF_KV_Q8_0>);
        default: return go(kv_write_kernel<AF_KV_Q4_0>);
    }
}

cudaError_t launch_kv_read(const KvRows& c, int n, const int* slots, int slot0, float* k, float* v, int64_t ld,
                           cudaStream_t s) {
    auto go = [&](auto kernel) { return launch_chained(kernel, dim3(ctas(n, kRows)), kThreads, 0, s, c, n, slots, slot0, k, v, ld); };
    switch (c.type) {
        case AF_F32: return go(kv_read_kernel<AF_F32>);
        case AF_F16: return go(kv_read_kernel<AF_F16>);
        case AF_KV_Q8_0: return go(kv_read_kernel<AF_KV_Q8_0>);
        default: return go(kv_read_kernel<AF_KV_Q4_0>);
    }
}

}  // namespace af

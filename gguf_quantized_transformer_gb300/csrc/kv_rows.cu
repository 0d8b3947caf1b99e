// Writing rows of keys and values into a cache of any type, and reading slots back as fp32 rows.
//
// A quantized cache holds, per 32 values along head_dim, an fp16 scale d and integer codes q, value d q:
//   Q8_0: d = fp16(max|v| / 127), q = clamp(round-half-away(v / d), -127, 127)
//   Q4_0: d = fp16(m / -8) with m the value of largest magnitude (the first on ties),
//         q = clamp(floor(v / d + 1/2), -8, 7)
// with the decisions those of exact arithmetic: with q a guess (v times 1 / d, rounded), q d has at most 8 + 11 bits and
// is an fp32 number, so r = v - q d comes out of one fused multiply-add exactly (v and q d are within a factor of two
// of each other, or q = 0), and comparing r with d / 2 corrects the guess.  A zero d gives zero codes.  A block that
// holds a NaN, or whose scale overflows fp16, gets a scale that makes all its values NaN: nothing non-finite is turned
// into a number.
//
// Both are bound by HBM.  A CTA takes kRows rows at a time and a thread four values of K and of V of each, all loads
// before the first use; the grid is a few CTAs per SM.  Data of earlier kernels is read through L2 (the kernels are
// launched with programmatic serialization).
#include <algorithm>

#include "draft.cuh"
#include "tma.cuh"

namespace af {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;
constexpr int kCtasPerSm = 6;

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

// Eight lanes (an aligned group of the warp) hold the 32 values of a block, four each.
template <int TYPE>
__device__ __forceinline__ void quantize_group(const float (&x)[4], unsigned group, int lane, int (&q)[4], __half& dh) {
    float amax = 0.f;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        amax = fmaxf(amax, fabsf(x[e]));
        nan |= x[e] != x[e];
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, o));
    nan = (__ballot_sync(group, nan) & group) != 0;
    if (TYPE == AF_KV_Q8_0) {
        dh = __float2half_rn(amax / 127.f);
    } else {
        float m = 0.f;
        bool has = false;
#pragma unroll
        for (int e = 3; e >= 0; e--)
            if (fabsf(x[e]) == amax) {
                m = x[e];
                has = true;
            }
        const unsigned who = __ballot_sync(group, has) & group;  // empty only when the block holds NaN alone
        m = __shfl_sync(group, m, who ? __ffs(who) - 1 : lane);
        dh = __float2half_rn(m / -8.f);
    }
    if (nan || (__half_as_ushort(dh) & 0x7C00) == 0x7C00) dh = __ushort_as_half((unsigned short)0x7FFF);
    const float d = fabsf(__half2float(dh)), rd = d == 0.f ? 0.f : __frcp_rn(d), h = 0.5f * d;
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, in the low bits
#pragma unroll
    for (int e = 0; e < 4; e++) {
        // the rounding is half away from zero on |v| for Q8_0, half up on v / d for Q4_0: half up on y / |d| either way
        const float y = TYPE == AF_KV_Q8_0 ? fabsf(x[e]) : (__half_as_ushort(dh) & 0x8000 ? -x[e] : x[e]);
        const float g = y * rd + kMagic;
        const float r = fmaf(-(g - kMagic), d, y);
        int v = __float_as_int(g) - 0x4B400000;
        v += (r >= h ? 1 : 0) - (r < -h ? 1 : 0);
        v = TYPE == AF_KV_Q8_0 ? min(v, 127) : min(max(v, -8), 7);
        if (TYPE == AF_KV_Q8_0 && x[e] < 0.f) v = -v;
        q[e] = d > 0.f ? v : 0;
    }
}

template <int TYPE>
__device__ __forceinline__ void store_group(void* base, __half* scales, int64_t cell, int D, int d0, const float (&x)[4],
                                            unsigned group, int lane) {
    if (TYPE == AF_F32) {
        *reinterpret_cast<float4*>((float*)base + cell * D + d0) = make_float4(x[0], x[1], x[2], x[3]);
    } else if (TYPE == AF_F16) {
        __half2 h[2] = {__floats2half2_rn(x[0], x[1]), __floats2half2_rn(x[2], x[3])};
        *reinterpret_cast<uint2*>((__half*)base + cell * D + d0) = *reinterpret_cast<const uint2*>(h);
    } else {
        int q[4];
        __half dh;
        quantize_group<TYPE>(x, group, lane, q, dh);
        if (TYPE == AF_KV_Q8_0) {
            const unsigned w = (unsigned)(q[0] & 255) | (unsigned)(q[1] & 255) << 8 | (unsigned)(q[2] & 255) << 16 |
                               (unsigned)(q[3] & 255) << 24;
            *reinterpret_cast<unsigned*>((uint8_t*)base + cell * D + d0) = w;
        } else {
            const unsigned w = (unsigned)(q[0] + 8) | (unsigned)(q[1] + 8) << 4 | (unsigned)(q[2] + 8) << 8 |
                               (unsigned)(q[3] + 8) << 12;
            *reinterpret_cast<unsigned short*>((uint8_t*)base + cell * (D / 2) + d0 / 2) = (unsigned short)w;
        }
        if ((lane & 7) == 0) scales[cell * (D / 32) + d0 / 32] = dh;
    }
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(KvRows c, const float* __restrict__ k, const float* __restrict__ v, int64_t ld, int n,
                    const int* __restrict__ slots, int slot0) {
    const int lane = threadIdx.x & 31;
    const unsigned group = 0xffu << (lane & 24);
    const int quads = c.KVH * c.D / 4;  // a multiple of 8
    pdl_launch_dependents();
    pdl_wait();
    for (int r0 = blockIdx.x * kRows; r0 < n; r0 += gridDim.x * kRows) {
        int slot[kRows];  // -1: not written; the same in every thread of the CTA
#pragma unroll
        for (int j = 0; j < kRows; j++) slot[j] = r0 + j >= n ? -1 : slots ? __ldcg(slots + r0 + j) : slot0 + r0 + j;
        if (slots) {
            unsigned again = 0;  // rows whose slot a later row names too: it belongs to that one
            for (int i = r0 + 1 + threadIdx.x; i < n; i += kThreads) {
                const int x = __ldcg(slots + i);
#pragma unroll
                for (int j = 0; j < kRows; j++) again |= (i > r0 + j && x == slot[j]) ? 1u << j : 0u;
            }
            again = cta_or(again);
#pragma unroll
            for (int j = 0; j < kRows; j++)
                if (slot[j] < 0 || slot[j] >= c.ctx || (again >> j & 1)) slot[j] = -1;
        }
        for (int i = threadIdx.x; i < quads; i += kThreads) {
            const int e0 = i * 4, g = e0 / c.D, d0 = e0 % c.D;
            float4 x[2][kRows];
#pragma unroll
            for (int j = 0; j < kRows; j++)
                if (slot[j] >= 0) {
                    x[0][j] = __ldcg(reinterpret_cast<const float4*>(k + (r0 + j) * ld + e0));
                    x[1][j] = __ldcg(reinterpret_cast<const float4*>(v + (r0 + j) * ld + e0));
                }
#pragma unroll
            for (int j = 0; j < kRows; j++)
                if (slot[j] >= 0) {
                    const int64_t cell = (int64_t)g * c.ctx + slot[j];
                    const float a[4] = {x[0][j].x, x[0][j].y, x[0][j].z, x[0][j].w};
                    const float b[4] = {x[1][j].x, x[1][j].y, x[1][j].z, x[1][j].w};
                    store_group<TYPE>(c.k, c.ks, cell, c.D, d0, a, group, lane);
                    store_group<TYPE>(c.v, c.vs, cell, c.D, d0, b, group, lane);
                }
        }
    }
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
    pdl_launch_dependents();
    pdl_wait();
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
}

unsigned ctas(int n) { return (unsigned)std::min((n + kRows - 1) / kRows, num_sms() * kCtasPerSm); }

}  // namespace

cudaError_t launch_kv_write(const KvRows& c, const float* k, const float* v, int64_t ld, int n, const int* slots,
                            int slot0, cudaStream_t s) {
    auto go = [&](auto kernel) { return launch_chained(kernel, dim3(ctas(n)), kThreads, 0, s, c, k, v, ld, n, slots, slot0); };
    switch (c.type) {
        case AF_F32: return go(kv_write_kernel<AF_F32>);
        case AF_F16: return go(kv_write_kernel<AF_F16>);
        case AF_KV_Q8_0: return go(kv_write_kernel<AF_KV_Q8_0>);
        default: return go(kv_write_kernel<AF_KV_Q4_0>);
    }
}

cudaError_t launch_kv_read(const KvRows& c, int n, const int* slots, int slot0, float* k, float* v, int64_t ld,
                           cudaStream_t s) {
    auto go = [&](auto kernel) { return launch_chained(kernel, dim3(ctas(n)), kThreads, 0, s, c, n, slots, slot0, k, v, ld); };
    switch (c.type) {
        case AF_F32: return go(kv_read_kernel<AF_F32>);
        case AF_F16: return go(kv_read_kernel<AF_F16>);
        case AF_KV_Q8_0: return go(kv_read_kernel<AF_KV_Q8_0>);
        default: return go(kv_read_kernel<AF_KV_Q4_0>);
    }
}

}  // namespace af

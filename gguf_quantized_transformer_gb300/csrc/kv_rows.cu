// Writing rows of keys and values into a cache of any type, and reading slots back as fp32 rows.
//
// A quantized cache holds, per 32 values along head_dim, an fp16 scale d and integer codes q, value d q:
//   Q8_0: d = fp16(max|v| / 127), q = clamp(round-half-away(v / d), -127, 127)
//   Q4_0: d = fp16(m / -8) with m the value of largest magnitude (the first on ties),
//         q = clamp(floor(v / d + 1/2), -8, 7)
// with the decisions those of exact arithmetic: the borders (k + 1/2) d have at most 19 significant bits, so they
// are fp32 numbers, and the correctly rounded fp32 quotient v / d of a v beside a border stays on its side (the
// distance of two fp32 numbers near v is at least 2^-24 of v, more than the half step 2^-25 .. 2^-24 that a
// quotient of that size is rounded by).  A zero d gives zero codes.  A block that holds a NaN, or whose scale
// overflows fp16, gets a scale that makes all its values NaN: nothing non-finite is turned into a number.
#include "draft.cuh"

namespace af {

namespace {

constexpr int kThreads = 256;

// Eight lanes (an aligned group of the warp) hold the 32 values of a block, four each.
struct Block4 {
    float x[4];
};

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
    if (nan) dh = __ushort_as_half((unsigned short)0x7FFF);
    const float d = __half2float(dh);
#pragma unroll
    for (int e = 0; e < 4; e++) {
        int v = 0;
        if (d != 0.f) {
            const float t = x[e] / d;
            if (TYPE == AF_KV_Q8_0) {
                const float f = floorf(fabsf(t));
                v = (int)f + (fabsf(t) - f >= 0.5f ? 1 : 0);
                v = v > 127 ? 127 : v;
                v = t < 0.f ? -v : v;
            } else {
                const float f = floorf(t);
                v = (int)f + (t - f >= 0.5f ? 1 : 0);
                v = v < -8 ? -8 : (v > 7 ? 7 : v);
            }
        }
        q[e] = v;
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

// One CTA per row of a grid-stride walk; a thread handles four values of K or V at a time.
template <int TYPE>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(KvRows c, const float* __restrict__ k, const float* __restrict__ v, int64_t ld, int n,
                    const int* __restrict__ slots, int slot0) {
    const int lane = threadIdx.x & 31;
    const unsigned group = 0xffu << (lane & 24);
    const int quads = c.KVH * c.D / 4;  // a multiple of 8
    for (int r = blockIdx.x; r < n; r += gridDim.x) {
        int slot = slot0 + r;
        if (slots) {
            slot = slots[r];
            if (slot < 0 || slot >= c.ctx) continue;  // uniform over the CTA
            // a slot that a later row names too belongs to that row
            bool again = false;
            for (int j = r + 1 + threadIdx.x; j < n; j += kThreads) again |= slots[j] == slot;
            if (__syncthreads_or(again)) continue;
        }
        for (int i = threadIdx.x; i < 2 * quads; i += kThreads) {
            const bool isv = i >= quads;
            const int e0 = (isv ? i - quads : i) * 4;
            const int g = e0 / c.D, d0 = e0 % c.D;
            const float4 f = *reinterpret_cast<const float4*>((isv ? v : k) + r * ld + e0);
            const float x[4] = {f.x, f.y, f.z, f.w};
            store_group<TYPE>(isv ? c.v : c.k, isv ? c.vs : c.ks, (int64_t)g * c.ctx + slot, c.D, d0, x, group, lane);
        }
    }
}

template <int TYPE>
__device__ __forceinline__ float4 load4(const void* base, const __half* scales, int64_t cell, int D, int d0) {
    if (TYPE == AF_F32) return *reinterpret_cast<const float4*>((const float*)base + cell * D + d0);
    if (TYPE == AF_F16) {
        const uint2 raw = *reinterpret_cast<const uint2*>((const __half*)base + cell * D + d0);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    const float d = __half2float(scales[cell * (D / 32) + d0 / 32]);
    if (TYPE == AF_KV_Q8_0) {
        const char4 q = *reinterpret_cast<const char4*>((const uint8_t*)base + cell * D + d0);
        return make_float4(d * (signed char)q.x, d * (signed char)q.y, d * (signed char)q.z, d * (signed char)q.w);
    }
    const unsigned w = *reinterpret_cast<const unsigned short*>((const uint8_t*)base + cell * (D / 2) + d0 / 2);
    return make_float4(d * ((int)(w & 15) - 8), d * ((int)(w >> 4 & 15) - 8), d * ((int)(w >> 8 & 15) - 8),
                       d * ((int)(w >> 12) - 8));
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(KvRows c, int n, const int* __restrict__ slots, int slot0, float* __restrict__ k,
                   float* __restrict__ v, int64_t ld) {
    const int quads = c.KVH * c.D / 4;
    for (int r = blockIdx.x; r < n; r += gridDim.x) {
        const int slot = slots ? slots[r] : slot0 + r;
        if (slot < 0 || slot >= c.ctx) continue;
        for (int i = threadIdx.x; i < 2 * quads; i += kThreads) {
            const bool isv = i >= quads;
            const int e0 = (isv ? i - quads : i) * 4;
            const int g = e0 / c.D, d0 = e0 % c.D;
            *reinterpret_cast<float4*>((isv ? v : k) + r * ld + e0) =
                load4<TYPE>(isv ? c.v : c.k, isv ? c.vs : c.ks, (int64_t)g * c.ctx + slot, c.D, d0);
        }
    }
}

}  // namespace

cudaError_t launch_kv_write(const KvRows& c, const float* k, const float* v, int64_t ld, int n, const int* slots,
                            int slot0, cudaStream_t s) {
    const unsigned blocks = (unsigned)(n < 65536 ? n : 65536);
    switch (c.type) {
        case AF_F32: kv_write_kernel<AF_F32><<<blocks, kThreads, 0, s>>>(c, k, v, ld, n, slots, slot0); break;
        case AF_F16: kv_write_kernel<AF_F16><<<blocks, kThreads, 0, s>>>(c, k, v, ld, n, slots, slot0); break;
        case AF_KV_Q8_0: kv_write_kernel<AF_KV_Q8_0><<<blocks, kThreads, 0, s>>>(c, k, v, ld, n, slots, slot0); break;
        default: kv_write_kernel<AF_KV_Q4_0><<<blocks, kThreads, 0, s>>>(c, k, v, ld, n, slots, slot0); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvRows& c, int n, const int* slots, int slot0, float* k, float* v, int64_t ld,
                           cudaStream_t s) {
    const unsigned blocks = (unsigned)(n < 65536 ? n : 65536);
    switch (c.type) {
        case AF_F32: kv_read_kernel<AF_F32><<<blocks, kThreads, 0, s>>>(c, n, slots, slot0, k, v, ld); break;
        case AF_F16: kv_read_kernel<AF_F16><<<blocks, kThreads, 0, s>>>(c, n, slots, slot0, k, v, ld); break;
        case AF_KV_Q8_0: kv_read_kernel<AF_KV_Q8_0><<<blocks, kThreads, 0, s>>>(c, n, slots, slot0, k, v, ld); break;
        default: kv_read_kernel<AF_KV_Q4_0><<<blocks, kThreads, 0, s>>>(c, n, slots, slot0, k, v, ld); break;
    }
    return cudaGetLastError();
}

}  // namespace af

// Attention for a tree of drafted tokens: node i of n sees the cached slots 0..past-1 and, of the slots
// past..past+n-1 that hold the nodes' own keys and values, those whose bit its mask row has:
//   out_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(q_i . k_j / sqrt(D)).
// A row that sees no slot gives zeros.
#include <math_constants.h>

#include "draft.cuh"

namespace af {

namespace {

// One warp per node: the lanes hold the mask words, and the walk up the parents sets a bit per ancestor.  A parent
// that is not an earlier node counts as -1, so that every walk ends.
__global__ void __launch_bounds__(256)
    tree_mask_kernel(const int* __restrict__ parent, int n, int pos0, unsigned* __restrict__ mask, int* __restrict__ pos) {
    __shared__ int up[kTreeMax];
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int p = parent[i];
        up[i] = p >= 0 && p < i ? p : -1;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, i = blockIdx.x * 8 + (threadIdx.x >> 5), words = (n + 31) / 32;
    if (i >= n) return;
    unsigned w = 0;
    int depth = -1;
    for (int j = i; j >= 0; j = up[j], depth++)
        if (j >> 5 == lane) w |= 1u << (j & 31);
    if (lane < words) mask[(int64_t)i * words + lane] = w;
    if (pos && lane == 0) pos[i] = pos0 + depth;
}

template <int TYPE>
__device__ __forceinline__ float cell_value(const void* base, const __half* scales, int64_t cell, int D, int d) {
    if (TYPE == AF_F32) return ((const float*)base)[cell * D + d];
    if (TYPE == AF_F16) return __half2float(((const __half*)base)[cell * D + d]);
    const float s = __half2float(scales[cell * (D / 32) + d / 32]);
    if (TYPE == AF_KV_Q8_0) return s * (float)((const int8_t*)base)[cell * D + d];
    const int b = ((const uint8_t*)base)[cell * (D / 2) + d / 2];
    return s * (float)((d & 1 ? b >> 4 : b & 15) - 8);
}

constexpr int kWarps = 8;

// One CTA per (node, head); the warps take the slots in turn, a lane owns D / 32 dims.
template <int TYPE, int D>
__global__ void __launch_bounds__(kWarps * 32) attn_tree_kernel(TreeArgs a) {
    constexpr int E = D / 32;
    __shared__ float sm_o[kWarps][D], sm_m[kWarps], sm_l[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x / a.H, h = blockIdx.x % a.H, g = h / (a.H / a.c.KVH);
    const int words = (a.n + 31) / 32;
    float q[E], o[E] = {};
#pragma unroll
    for (int e = 0; e < E; e++) q[e] = a.q[i * a.ldq + h * D + lane + 32 * e] * rsqrtf((float)D);
    float m = -CUDART_INF_F, l = 0.f;
    for (int j = warp; j < a.past + a.n; j += kWarps) {
        const int t = j - a.past;
        if (t >= 0 && !(a.mask[(int64_t)i * words + (t >> 5)] >> (t & 31) & 1)) continue;
        const int64_t cell = (int64_t)g * a.c.ctx + j;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; e++) s += q[e] * cell_value<TYPE>(a.c.k, a.c.ks, cell, D, lane + 32 * e);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < E; e++) o[e] = o[e] * f + p * cell_value<TYPE>(a.c.v, a.c.vs, cell, D, lane + 32 * e);
        m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; e++) sm_o[warp][lane + 32 * e] = o[e];
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float mx = -CUDART_INF_F, num = 0.f, den = 0.f;
        for (int w = 0; w < kWarps; w++) mx = fmaxf(mx, sm_m[w]);
        for (int w = 0; w < kWarps; w++) {
            if (sm_l[w] == 0.f) continue;
            const float f = expf(sm_m[w] - mx);
            num += f * sm_o[w][d];
            den += f * sm_l[w];
        }
        a.out[i * a.ldo + h * D + d] = den == 0.f ? 0.f : num / den;
    }
}

template <int TYPE>
cudaError_t go(const TreeArgs& a, cudaStream_t s) {
    if (a.c.D == 64)
        attn_tree_kernel<TYPE, 64><<<a.n * a.H, kWarps * 32, 0, s>>>(a);
    else
        attn_tree_kernel<TYPE, 128><<<a.n * a.H, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_mask(const int* parent, int n, int pos0, unsigned* mask, int* pos, cudaStream_t s) {
    tree_mask_kernel<<<(n + 7) / 8, 256, 0, s>>>(parent, n, pos0, mask, pos);
    return cudaGetLastError();
}

size_t attn_tree_ws_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_attn_tree(const TreeArgs& a, cudaStream_t s) {
    switch (a.c.type) {
        case AF_F32: return go<AF_F32>(a, s);
        case AF_F16: return go<AF_F16>(a, s);
        case AF_KV_Q8_0: return go<AF_KV_Q8_0>(a, s);
        default: return go<AF_KV_Q4_0>(a, s);
    }
}

}  // namespace af

// Paged attention: the join of pieces that several CTAs hold, and the dispatch by cache type (attn_paged_impl.cuh).
#include "attn_paged_impl.cuh"

namespace af {

template <>
cudaError_t launch_attn_paged_type<AF_F32>(const PagedArgs&, int, cudaStream_t);
template <>
cudaError_t launch_attn_paged_type<AF_F16>(const PagedArgs&, int, cudaStream_t);
template <>
cudaError_t launch_attn_paged_type<AF_KV_Q8_0>(const PagedArgs&, int, cudaStream_t);
template <>
cudaError_t launch_attn_paged_type<AF_KV_Q4_0>(const PagedArgs&, int, cudaStream_t);

namespace {

constexpr int kJoinWarps = 16;

// Block b joins the item that begins in CTA b and goes on in others: piece 1 of b, then piece 0 of b + 1 and so on up to the
// CTA in which it ends.  Two warps per head take the pieces in turn, their sums are added in order.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(PagedArgs a, int ctas, int heads) {
    __shared__ int sm_last;
    __shared__ float4 sm_num[kJoinWarps][32];
    __shared__ float2 sm_den[kJoinWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
    const PagedPiece* info = reinterpret_cast<const PagedPiece*>(a.ws + (size_t)ctas * 2 * paged_piece_floats(D));
    pdl_launch_dependents();
    pdl_wait();
    const int4 me = __ldcg(reinterpret_cast<const int4*>(info + 2 * b + 1));
    if (!me.z) return;
    if (tid == 0) sm_last = ctas - 1;
    __syncthreads();
    for (int x = b + 1 + tid; x < ctas; x += kJoinWarps * 32) {
        const int4 y = __ldcg(reinterpret_cast<const int4*>(info + 2 * x));
        if (y.z && y.w) atomicMin(&sm_last, x);
    }
    __syncthreads();
    const int n = sm_last - b + 1;  // pieces, those of CTAs that had no part of any item among them
    const int per = kJoinWarps / heads, hh = warp / per, sub = warp % per;
    const int G = a.H / a.c.KVH, HT = (G + heads - 1) / heads, g = me.y / HT, head = (me.y - g * HT) * heads + hh;
    auto base = [&](int i) { return a.ws + (size_t)(2 * (b + i) + (i ? 0 : 1)) * paged_piece_floats(D); };
    auto used = [&](int i) { return i == 0 || __ldcg(&info[2 * (b + i)].used) != 0; };
    auto stat = [&](int i) {
        return used(i) ? __ldcg(reinterpret_cast<const float2*>(base(i) + kPagedHeads * D) + hh) : make_float2(-CUDART_INF_F, 0.f);
    };
    const bool in = hh < heads && head < G;
    float m = -CUDART_INF_F;
    bool saw = false;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
    if (in) {
        for (int i = lane; i < n; i += 32) {
            const float2 ml = stat(i);
            m = fmaxf(m, ml.x);
            saw |= __float_as_uint(ml.y) != 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        saw = __any_sync(0xffffffffu, saw);
        const int d = 4 * lane < D ? 4 * lane : 0;
        for (int i0 = 0; i0 * per < n; i0 += 32) {  // this warp's pieces sub + per * (i0 + ..)
            const int mine = (i0 + lane) * per + sub;
            float2 ml = make_float2(-CUDART_INF_F, 0.f);
            if (mine < n) ml = stat(mine);
            const bool none = ml.x == -CUDART_INF_F && ml.y == 0.f;
            const float f = none ? 0.f : ex2t(ml.x - m);
            den += none ? 0.f : f * ml.y;
            const unsigned live = __ballot_sync(0xffffffffu, !none);
            for (int k0 = 0; k0 < 32 && (i0 + k0) * per + sub < n; k0 += 8) {
                float4 v[8];
#pragma unroll
                for (int k = 0; k < 8; k++)
                    v[k] = live >> (k0 + k) & 1 ? __ldcg(reinterpret_cast<const float4*>(base((i0 + k0 + k) * per + sub) + hh * D + d))
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float w = __shfl_sync(0xffffffffu, f, k0 + k);
                    num.x += w * v[k].x, num.y += w * v[k].y, num.z += w * v[k].z, num.w += w * v[k].w;
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    }
    sm_num[warp][lane] = num;
    if (lane == 0) sm_den[warp] = make_float2(den, 0.f);
    __syncthreads();
    if (!in || sub || 4 * lane >= D) return;
    for (int i = 1; i < per; i++) {
        const float4 y = sm_num[warp + i][lane];
        num.x += y.x, num.y += y.y, num.z += y.z, num.w += y.w;
        den += sm_den[warp + i].x;
    }
    const float inv = den != 0.f ? 1.f / den : saw ? CUDART_NAN_F : 0.f;
    *reinterpret_cast<float4*>(a.out + (int64_t)me.x * a.ldo + (int64_t)(g * G + head) * D + 4 * lane) =
        make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
}

}  // namespace

size_t attn_paged_ws_bytes(int D) {
    return paged_ws_floats(num_sms(), D) * sizeof(float);
}

cudaError_t launch_attn_paged(const PagedArgs& a, cudaStream_t s) {
    const int ctas = num_sms(), heads = a.H / a.c.KVH > 4 ? 8 : 4;
    cudaError_t e;
    switch (a.c.type) {
        case AF_F32: e = launch_attn_paged_type<AF_F32>(a, ctas, s); break;
        case AF_F16: e = launch_attn_paged_type<AF_F16>(a, ctas, s); break;
        case AF_KV_Q8_0: e = launch_attn_paged_type<AF_KV_Q8_0>(a, ctas, s); break;
        default: e = launch_attn_paged_type<AF_KV_Q4_0>(a, ctas, s); break;
    }
    if (e) return e;
    if (a.c.D == 64) return launch_chained(paged_join_kernel<64>, dim3(ctas - 1), kJoinWarps * 32, 0, s, a, ctas, heads);
    return launch_chained(paged_join_kernel<128>, dim3(ctas - 1), kJoinWarps * 32, 0, s, a, ctas, heads);
}

}  // namespace af

// Attention for a tree of drafted tokens: node i of n sees the cached slots 0..past-1 and, of the slots
// past..past+n-1 that hold the nodes' own keys and values, those whose bit its mask row has:
//   out_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(q_i . k_j / sqrt(D)).
// A row that sees no slot gives zeros; one whose scores are all -infinity has no softmax and gives NaN.
//
// The rows of a kv head are its n nodes times the G heads of its group (row = node G + head), so that every cached
// byte is read once for all of them.  Split-KV: CTA (split, kv head, row tile of 16 MT rows) walks its range of
// slots once; inside it every warp takes its own stages of KS slots through a private cp.async ring, with its own
// running maximum, sum and output (mma.sync fragments in registers), no CTA barrier in the loop, and the warps'
// states are joined at the end.  With several splits the partials are joined by a second kernel in split order.
//
// Scores and output on the tensor cores at fp32-level precision:
//  - q (scaled by log2 e / sqrt(D): p = 2^(s - m)) is split into two parts of 11 bits, fp16 (scaled by a power of
//    two per row, so no magnitude overflows) or tf32; so is p.
//  - fp16 cache: K and V are operands as they are; two products each (hi and lo).
//  - Q8_0 / Q4_0: the integer codes are exact fp16 operands.  A key's scale multiplies its fp32 partial score of
//    each 32-value block; a value's scale multiplies p, per block, before p is split.  Both stay in fp16's range: a
//    thread takes its slots' scales times 2^-ev, which brings them near 1, and p times 2^(ev - ov), where the row's
//    exponent ov follows the largest p 2^ev of the slots that the row sees.  A stage in which a thread's scales are
//    more than 2^8 apart (one large scale, hidden or not, would leave the others few bits) is walked again for the
//    smaller ones.
//  - fp32 cache: tf32 parts of K and V too, three products (the dropped lo lo product is 2^-21 relative at most).
// The tensor cores cut their fp32 sums (every product takes up to 2^-23 of the sum, towards zero: one sum over a warp's 80
// stages of fp32 slots was off by 1.1e-5 of the result's norm), so a stage's output starts from zero and is added,
// rounded, to the walk's: 1.2e-7.  (fp32, 1 and 4 tokens over 30000 slots: 48.3 and 65.9 us, 45.2 and 55.7 with one sum.)
// So do scores every 32 dims, small lo products first (3 nodes over 6000 fp32 slots: 4e-7, 2.1e-6 with one sum over the head).
// The reference maximum of the softmax moves only when a score exceeds it by more than 4 (in powers of two); p
// carries a factor 2^8 so that small p keep their low part above fp16's subnormal step.  Sums are fp32.
//
// A call of up to 8 rows (MT = 0) puts the hi parts of q and p into rows 0-7 of the 16-row tile and the lo parts into rows
// 8-15: one product instead of two, whose halves are added (one token over 30000 Q8_0 slots: 28.4 us with two products,
// 23.0 with one; fp32 64.9 and 48.7).
//
// Hidden slots: a masked score is -inf (a select, so NaN does not survive); in the groups of slots that hold nodes,
// non-finite values are taken out of the product and added element by element to the rows that see them.
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "draft.cuh"
#include "tma.cuh"

namespace af {

namespace {

// One warp per node: the lanes hold the mask words, and the walk up the parents sets a bit per ancestor.  A parent
// that is not an earlier node counts as -1, so that every walk ends.
__global__ void __launch_bounds__(256)
    tree_mask_kernel(const int* __restrict__ parent, int n, int pos0, unsigned* __restrict__ mask, int* __restrict__ pos) {
    __shared__ int up[kTreeMax];
    pdl_launch_dependents();
    pdl_wait();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int p = __ldcg(parent + i);
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

// ---------------------------------------------------------------- building blocks

constexpr float kLog2eT = 1.4426950408889634f;
constexpr float kLazyT = 4.f;  // powers of two by which a score may exceed the reference maximum
constexpr float kBiasT = 8.f;  // p = 2^(s - m + kBiasT): at most 2^12
constexpr float kNoRefT = -1000.f;  // a row's exponent of the output before it has one

__device__ __forceinline__ float ex2t(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 ldsm4t(uint32_t a) {
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// The same onto zero
__device__ __forceinline__ void mma16z(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma8z(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}
// o += c, rounded: a stage's sum joins the walk's
__device__ __forceinline__ void add4(float (&o)[4], const float (&c)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 x = add2(make_float2(o[i], o[i + 1]), make_float2(c[i], c[i + 1]));
        o[i] = x.x, o[i + 1] = x.y;
    }
}
__device__ __forceinline__ uint32_t tf32_of(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
// x = hi + lo in two tf32 parts
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = tf32_of(x);
    lo = tf32_of(x - __uint_as_float(hi));
}
// The same for a value of the cache, whose hi part is cut, not rounded: rounded, fp32's largest numbers would be infinities,
// which times a zero weight are NaN.  lo is then up to 2^-10 of x and off by 2^-22.  (One token over 30000 fp32 slots
// 45.2 us, 51.9 with rounded parts: the cut is a plain logic instruction.)
__device__ __forceinline__ void cut_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(x) & 0xFFFFE000u;
    lo = tf32_of(x - __uint_as_float(hi));
}
// (a, b) = hi + lo in two fp16 parts each
__device__ __forceinline__ void split_h2(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 r = fma2(__half22float2(h), both(-1.f), make_float2(a, b));
    const __half2 l = __floats2half2_rn(r.x, r.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}
// two halves of `magic + code` minus `off`: the codes as fp16
__device__ __forceinline__ uint32_t hsub2u(uint32_t x, uint32_t off) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&off));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// non-finite halves of x become 0; `bad` is set if there were any
__device__ __forceinline__ uint32_t finite_h2(uint32_t x, bool& bad) {
    const bool lo = (x & 0x7C00u) == 0x7C00u, hi = (x & 0x7C000000u) == 0x7C000000u;
    bad |= lo | hi;
    return x & ((lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u));
}

// Slots a warp takes at a time and warps of a CTA.  Of up to 8 rows over codes twelve warps of 168 registers fit (one token
// over 30000 Q8_0 slots 22.5 us, 24.0 with ten); with 16 rows a stage's sums need more (4 tokens 29.4 us, 34.5 with twelve).
__host__ __device__ constexpr int tree_stage(int type, int mt) {
    return (type == AF_KV_Q8_0 || type == AF_KV_Q4_0) && mt <= 1 ? 32 : 16;
}
__host__ __device__ constexpr int tree_warps(int type, int D, int mt) {
    return type == AF_F32 && D == 128 ? 6 : (type == AF_KV_Q8_0 || type == AF_KV_Q4_0) && mt == 0 ? 12 : 8;
}

template <int TYPE, int D, int MT>
struct TreeCfg {
    static constexpr bool QUANT = TYPE == AF_KV_Q8_0 || TYPE == AF_KV_Q4_0;
    static constexpr bool PACK = MT == 0;
    static constexpr int ROWS = PACK ? 8 : 16 * MT;
    static constexpr int NB = D / 32;                                             // 32-value blocks of a head
    static constexpr int RB = TYPE == AF_F32 ? 4 * D : TYPE == AF_F16 ? 2 * D : TYPE == AF_KV_Q8_0 ? D : D / 2;  // row bytes
    static constexpr int SB = QUANT ? 2 * NB : 0;                                 // scale bytes of a row
    static constexpr int KS = tree_stage(TYPE, MT);                               // slots per stage
    static constexpr int NW = tree_warps(TYPE, D, MT);                            // warps
    static constexpr int OV = KS * RB, OKS = 2 * KS * RB, OVS = OKS + KS * SB;    // V, K scales, V scales in a stage
    static constexpr int STAGE = 2 * KS * (RB + SB);
    static constexpr int RING = (QUANT ? 216 : 192) * 1024;
    static constexpr int NST = RING / (NW * STAGE) < 4 ? RING / (NW * STAGE) : 4;  // stages of a warp
    static_assert(NST >= 2, "a stage in flight while one is read");
    static constexpr int DP = D + (TYPE == AF_F16 ? 8 : 4);                       // padded output row of the join
    static constexpr int KQ = TYPE == AF_F32 ? D / 8 : D / 16;                    // mma steps along a head
    // 16-byte chunk permutation of row `key`, so that the fragment loads of a warp meet all banks
    static __device__ __forceinline__ int swk(int key) {
        if (TYPE == AF_F32) return key & 1;
        if (TYPE == AF_F16) return (key & 1) << 2;
        if (TYPE == AF_KV_Q8_0) return D == 128 ? (key & 3) << 1 : (key & 2);
        return D == 128 ? (key >> 1) & 3 : (key >> 2) & 1;
    }
    static __device__ __forceinline__ int swv(int key) {
        if (TYPE == AF_F32) return ((key >> 1) & 3) << 1;
        if (TYPE == AF_F16) return key & 7;
        if (TYPE == AF_KV_Q8_0) return D == 128 ? ((key >> 1) & 3) << 1 : (key & 2);
        return D == 128 ? (key >> 1) & 3 : (key >> 2) & 1;
    }
    // dim of the output fragment's column m (0..7) of n-tile t
    static __device__ __forceinline__ int odim(int t, int m) {
        return TYPE == AF_F16 ? 8 * t + m : 32 * (t >> 2) + 4 * m + (t & 3);
    }
};
template <int TYPE, int D, int MT>
constexpr int tree_q_bytes() {
    return TreeCfg<TYPE, D, MT>::KQ * 32 * 16 * (MT ? 2 * MT : 1);
}
template <int TYPE, int D, int MT>
constexpr int tree_smem() {
    using C = TreeCfg<TYPE, D, MT>;
    constexpr int ring = C::NW * C::NST * C::STAGE, join = C::NW * C::ROWS * (C::DP + 2) * 4;
    return tree_q_bytes<TYPE, D, MT>() + (ring > join ? ring : join);
}

// A lane's scales of a stage (slot `lane`, K and V) on their way through registers: copies of 4 or 8 bytes would go through
// L1, which may hold what an earlier kernel of the chain has overwritten since.
struct TreeScales {
    uint2 k, v;
    uint32_t dst = 0;  // 0: none
};
template <int TYPE, int D, int MT>
__device__ __forceinline__ void tree_put(const TreeScales& s, int lane) {
    using C = TreeCfg<TYPE, D, MT>;
    if (!C::QUANT || !s.dst || (C::KS < 32 && lane >= C::KS)) return;
    const uint32_t k = s.dst + C::OKS + lane * C::SB, v = s.dst + C::OVS + lane * C::SB;
    if (C::SB == 8) {
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(k), "r"(s.k.x), "r"(s.k.y) : "memory");
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(v), "r"(s.v.x), "r"(s.v.y) : "memory");
    } else {
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(k), "r"(s.k.x) : "memory");
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(v), "r"(s.v.x) : "memory");
    }
}

// One stage of a warp: slots [key0, key0 + KS), of which those below `end` are read.  The scales come back in `s`, for
// tree_put once they are there.
template <int TYPE, int D, int MT>
__device__ __forceinline__ void tree_issue(const KvRows& c, int64_t row0, int key0, int end, uint32_t dst, int lane,
                                           TreeScales& s) {
    using C = TreeCfg<TYPE, D, MT>;
    constexpr int CPR = C::RB / 16;
    const uint8_t* k = (const uint8_t*)c.k + row0 * C::RB;
    const uint8_t* v = (const uint8_t*)c.v + row0 * C::RB;
#pragma unroll
    for (int i = 0; i < C::KS * CPR / 32; i++) {
        const int idx = i * 32 + lane, key = idx / CPR, ch = idx % CPR;
        const bool in = key0 + key < end;
        const int64_t off = in ? (int64_t)(key0 + key) * C::RB + ch * 16 : 0;
        cp16(dst + key * C::RB + ((ch ^ C::swk(key)) << 4), k + off, in);
        cp16(dst + C::OV + key * C::RB + ((ch ^ C::swv(key)) << 4), v + off, in);
    }
    if (C::QUANT) {
        s.dst = dst;
        s.k = s.v = make_uint2(0u, 0u);
        if ((C::KS == 32 || lane < C::KS) && key0 + lane < end) {
            const int64_t off = (row0 + key0 + lane) * C::SB;
            if (C::SB == 8) {
                s.k = __ldcg(reinterpret_cast<const uint2*>((const uint8_t*)c.ks + off));
                s.v = __ldcg(reinterpret_cast<const uint2*>((const uint8_t*)c.vs + off));
            } else {
                s.k.x = __ldcg(reinterpret_cast<const unsigned*>((const uint8_t*)c.ks + off));
                s.v.x = __ldcg(reinterpret_cast<const unsigned*>((const uint8_t*)c.vs + off));
            }
        }
    }
}

// Scales of slots key (low half) and key + 1 (key even) by block; a: address of slot key's scales, [slot][block]
template <int NB>
__device__ __forceinline__ void load_scales(uint32_t a, uint32_t (&d)[NB]) {
    uint32_t w[NB];
    if (NB == 4) {
        const uint4 r = lds128(a);
        w[0] = r.x, w[1] = r.y, w[NB - 2] = r.z, w[NB - 1] = r.w;
    } else {
        const uint2 r = lds64(a);
        w[0] = r.x, w[NB - 1] = r.y;
    }
#pragma unroll
    for (int b = 0; b < NB; b++) d[b] = __byte_perm(w[b / 2], w[NB / 2 + b / 2], b & 1 ? 0x7632 : 0x5410);
}
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// The value of (key, dim) of a stage's V, for the element-by-element path.
template <int TYPE, int D, int MT>
__device__ __forceinline__ float stage_value(uint32_t st, int key, int d) {
    using C = TreeCfg<TYPE, D, MT>;
    const uint32_t row = st + C::OV + key * C::RB;
    auto at = [&](int byte) { return row + ((((byte >> 4) ^ C::swv(key)) << 4) | (byte & 15)); };
    if (TYPE == AF_F32) return __uint_as_float(lds32(at(4 * d)));
    if (TYPE == AF_F16) return __half2float(__ushort_as_half((unsigned short)lds16(at(2 * d))));
    const float s = __half2float(__ushort_as_half((unsigned short)lds16(st + C::OVS + key * C::SB + 2 * (d >> 5))));
    if (TYPE == AF_KV_Q8_0) {
        const uint32_t w = lds16(at(d & ~1));
        return s * (float)(int8_t)(d & 1 ? w >> 8 : w & 255);
    }
    const uint32_t w = lds16(at((d >> 1) & ~1));
    return s * (float)((int)(w >> (4 * (d & 3)) & 15) - 8);
}

template <int TYPE, int D, int MT_>
__global__ void __launch_bounds__(TreeCfg<TYPE, D, MT_>::NW * 32, 1) attn_tree_kernel(TreeArgs a, int splits) {
    using C = TreeCfg<TYPE, D, MT_>;
    constexpr bool PACK = C::PACK;
    constexpr int MT = PACK ? 1 : MT_, NH = PACK ? 1 : 2;  // row tiles, rows of a tile per thread
    constexpr int QP = PACK ? 1 : 2;                       // fragments of q per step and row tile
    constexpr int NW = C::NW, NT = D / 8, KS = C::KS, GT = KS / 8, NB = C::NB, ROWS = C::ROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sm_rowf[ROWS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, j = lane >> 2;
    const int G = a.H / a.c.KVH, R = a.n * G, keys = a.past + a.n;
    const int split = blockIdx.x, g = blockIdx.y, r0 = blockIdx.z * ROWS;
    const int stages = (keys + KS - 1) / KS;
    const int st0 = (int)((int64_t)stages * split / splits), st1 = (int)((int64_t)stages * (split + 1) / splits);
    const int64_t row0 = (int64_t)g * a.c.ctx;
    const uint32_t sq = smem_u32(smem), ring = sq + tree_q_bytes<TYPE, D, MT_>() + warp * C::NST * C::STAGE;

    pdl_launch_dependents();
    pdl_wait();  // q, the mask and the cache are written by earlier kernels
    // ---- the first stages are on their way while q is prepared
    TreeScales first[C::NST - 1];
#pragma unroll
    for (int i = 0; i < C::NST - 1; i++) {
        const int st = st0 + warp + i * NW;
        if (st < st1) tree_issue<TYPE, D, MT_>(a.c, row0, st * KS, keys, ring + i * C::STAGE, lane, first[i]);
        cp_commit();
    }

    // ---- q fragments: a warp scales and splits a row; lane l holds dims 4l..4l+3
    constexpr int RPW = (ROWS + NW - 1) / NW;
    float4 qin[RPW];
#pragma unroll
    for (int i = 0; i < RPW; i++) {
        const int r = warp + i * NW;
        qin[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < ROWS && r0 + r < R && lane < D / 4) {
            const int node = (r0 + r) / G, head = g * G + (r0 + r) % G;
            qin[i] = __ldcg(reinterpret_cast<const float4*>(a.q + (int64_t)node * a.ldq + (int64_t)head * D + 4 * lane));
        }
    }
#pragma unroll
    for (int ri = 0; ri < RPW; ri++) {
        const int r = warp + ri * NW;
        if (r >= ROWS) break;
        const float sc = rsqrtf((float)D) * kLog2eT;
        float x[4] = {qin[ri].x * sc, qin[ri].y * sc, qin[ri].z * sc, qin[ri].w * sc};
        if (TYPE != AF_F32) {  // a power of two brings the row's largest value to [1, 2)
            float mx = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            int e = (int)(__float_as_uint(mx) >> 23) - 127;
            e = e < -100 ? -100 : (e > 126 ? 126 : e);  // (0, subnormal; infinite: the row becomes NaN either way)
            const float down = __uint_as_float((unsigned)(127 - e) << 23);
#pragma unroll
            for (int i = 0; i < 4; i++) x[i] *= down;
            if (lane == 0) sm_rowf[r] = __uint_as_float((unsigned)(127 + e) << 23);
        }
        if (lane < D / 4) {
            const int mt = r >> 4, rr = r & 15, b = lane >> 3, cc = (lane & 7) >> 1, par = lane & 1;
            const uint32_t lane_off = (uint32_t)((rr & 7) * 4 + cc) * 16, hi8 = (uint32_t)(rr >> 3);
            // register of half h: rows 8-15 are the second of a pair, of the same part or (PACK) the lo part
            auto frag = [&](int step, int h, int part) {
                return sq + (uint32_t)((step * MT + mt) * QP + (PACK ? 0 : part)) * 512 + lane_off + (2 * h + (PACK ? part : hi8)) * 4;
            };
            if (TYPE == AF_F32) {
#pragma unroll
                for (int i = 0; i < 4; i++) {  // dim 8 cc + 2 s + h: register 2 h + (row >= 8) of step 4 b + s
                    uint32_t hi, lo;
                    split_tf32(x[i], hi, lo);
                    const int step = 4 * b + 2 * par + (i >> 1);
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(frag(step, i & 1, 0)), "r"(hi) : "memory");
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(frag(step, i & 1, 1)), "r"(lo) : "memory");
                }
            } else {
                uint32_t hi[2], lo[2];
                split_h2(x[0], x[1], hi[0], lo[0]);
                split_h2(x[2], x[3], hi[1], lo[1]);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    // dim 8 cc + i of its half: Q4_0 pairs dims 4 apart (their nibbles share a mask), else neighbours
                    const int dd = 4 * par + i;
                    const int s = TYPE == AF_KV_Q4_0 ? (dd & 3) >> 1 : dd >> 2, h = TYPE == AF_KV_Q4_0 ? dd & 1 : (dd >> 1) & 1;
                    const int e = TYPE == AF_KV_Q4_0 ? dd >> 2 : dd & 1;
                    const unsigned short vh = (unsigned short)(hi[i >> 1] >> (16 * (i & 1)));
                    const unsigned short vl = (unsigned short)(lo[i >> 1] >> (16 * (i & 1)));
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(frag(2 * b + s, h, 0) + 2 * e), "h"(vh) : "memory");
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(frag(2 * b + s, h, 1) + 2 * e), "h"(vl) : "memory");
                }
            }
        }
    }
    __syncthreads();
    float rowf[MT][NH];
    const unsigned* mrow[MT][NH];  // mask words of this thread's rows
    const int words = (a.n + 31) / 32;
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int h = 0; h < NH; h++) {
            const int r = mt * 16 + h * 8 + j;
            rowf[mt][h] = TYPE == AF_F32 ? 1.f : sm_rowf[r];
            mrow[mt][h] = r0 + r < R ? a.mask + (int64_t)((r0 + r) / G) * words : nullptr;
        }
    // bit i: the row sees slot key0 + i of the cache
    auto window = [&](int mt, int h, int key0) {
        const int t = key0 - a.past, w = t >> 5;  // t < 0: slots of the past, which every row sees
        const unsigned* m = mrow[mt][h];
        const unsigned lo = w < 0 ? ~0u : (m && w < words ? __ldcg(m + w) : 0u);
        const unsigned hi = w + 1 < 0 ? ~0u : (m && w + 1 < words ? __ldcg(m + w + 1) : 0u);
        const unsigned x = __funnelshift_r(lo, hi, t & 31);
        return t + 32 <= a.n ? x : (t >= a.n ? 0u : x & ((1u << (a.n - t)) - 1u));  // nothing behind the last node
    };

    float o[MT][NT][4] = {}, m_ref[MT][NH], l[MT][NH] = {};
    // Quantized: this thread's scales are taken times 2^-ev (above vlim / 2^8 and up to vlim = 2^(ev + 2)), p times 2^(ev - ov),
    // so that the output is held times 2^-ov and the thread's part of the sum times 2^(ev - ov).
    float ov[MT][NH], ev = C::QUANT ? -15.f : 0.f, vlim = 0x1p-13f;
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int h = 0; h < NH; h++) m_ref[mt][h] = -CUDART_INF_F, ov[mt][h] = C::QUANT ? kNoRefT : 0.f;

    int slot = 0;
    TreeScales scales;
#pragma unroll
    for (int i = 0; i < C::NST - 1; i++) tree_put<TYPE, D, MT_>(first[i], lane);
    constexpr unsigned kAll = (1u << (2 * GT)) - 1;
    unsigned todo = kAll;  // quantized: bit 2 t + i: this thread's slot 8 t + 2 c + i has to be walked yet
    bool again = false;    // this stage has been walked and is so once more, for slots that are left
    for (int st = st0 + warp; st < st1;) {
        if (!again) {
            cp_wait<C::NST - 2>();
            tree_put<TYPE, D, MT_>(scales, lane);  // of the stage issued last, with NST = 2 this one
            __syncwarp();  // every lane's copies of this stage have landed, and every lane is done with the previous one
            asm volatile("" ::: "memory");
            // the previous stage's slot takes the stage NST - 1 ahead
            const int nx = st + (C::NST - 1) * NW, ns = slot == 0 ? C::NST - 1 : slot - 1;
            scales.dst = 0;
            if (nx < st1) tree_issue<TYPE, D, MT_>(a.c, row0, nx * KS, keys, ring + ns * C::STAGE, lane, scales);
            cp_commit();
        }
        const uint32_t base = ring + slot * C::STAGE;
        const int key0 = st * KS;
        const uint32_t vb0 = base + C::OV;
        const bool nodes = key0 + KS > a.past;  // slots of nodes, or behind the last one
        unsigned see[MT][NH] = {};
        if (nodes)
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int h = 0; h < NH; h++) see[mt][h] = window(mt, h, key0);
        // ---- scores of the stage's slots: tile t, columns 2c and 2c + 1, are slots 8 t + 2 c, + 1
        float s[MT][GT][4] = {};
        if constexpr (C::QUANT) {
            uint32_t dk[GT][NB];
#pragma unroll
            for (int t = 0; t < GT; t++) load_scales<NB>(base + C::OKS + (t * 8 + 2 * c) * C::SB, dk[t]);
#pragma unroll
            for (int b = 0; b < NB; b++) {
                uint32_t kw[GT][4];
#pragma unroll
                for (int t = 0; t < GT; t++) {
                    const int key = t * 8 + j;
                    if (TYPE == AF_KV_Q8_0) {
                        const int byte = 32 * b + 8 * c;
                        uint2 w = lds64(base + key * C::RB + ((((byte >> 4) ^ C::swk(j)) << 4) | (byte & 15)));
                        w.x ^= 0x80808080u, w.y ^= 0x80808080u;
                        kw[t][0] = hsub2u(__byte_perm(w.x, 0x64646464u, 0x4140), 0x64806480u);
                        kw[t][1] = hsub2u(__byte_perm(w.x, 0x64646464u, 0x4342), 0x64806480u);
                        kw[t][2] = hsub2u(__byte_perm(w.y, 0x64646464u, 0x4140), 0x64806480u);
                        kw[t][3] = hsub2u(__byte_perm(w.y, 0x64646464u, 0x4342), 0x64806480u);
                    } else {
                        const uint32_t w = lds32(base + key * C::RB + ((b ^ C::swk(j)) << 4) + 4 * c);
#pragma unroll
                        for (int i = 0; i < 4; i++) kw[t][i] = hsub2u(((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u, 0x64086408u);
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
                    float p[GT][4] = {};
#pragma unroll
                    for (int i = PACK ? 2 : 0; i < 4; i++) {  // q's lo parts (steps 0 and 1), then its hi parts
                        const int e = i & 1;
                        const uint4 q = lds128(sq + ((2 * b + e) * MT + mt) * QP * 512 + (i < 2 ? 512 : 0) + lane * 16);
#pragma unroll
                        for (int t = 0; t < GT; t++) mma16(p[t], q, kw[t][2 * e], kw[t][2 * e + 1]);
                    }
#pragma unroll
                    for (int t = 0; t < GT; t++) {
                        const float2 dd = __half22float2(as_h2(dk[t][b]));
#pragma unroll
                        for (int h = 0; h < 2; h++) {  // (PACK: the lo parts' scores too, added below)
                            const float2 x = fma2(dd, make_float2(p[t][2 * h], p[t][2 * h + 1]),
                                                  make_float2(s[mt][t][2 * h], s[mt][t][2 * h + 1]));
                            s[mt][t][2 * h] = x.x, s[mt][t][2 * h + 1] = x.y;
                        }
                    }
                }
            }
        } else if constexpr (TYPE == AF_F16) {
#pragma unroll
            for (int b = 0; b < NB; b++) {
                uint4 kw[GT];
#pragma unroll
                for (int t = 0; t < GT; t++) kw[t] = lds128(base + (t * 8 + j) * C::RB + (((4 * b + c) ^ C::swk(j)) << 4));
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
                    float p[GT][4] = {};  // of the block: its sum starts from zero, as the output's does
#pragma unroll
                    for (int i = PACK ? 2 : 0; i < 4; i++) {  // q's lo parts (steps 0 and 1), then its hi parts
                        const int e = i & 1;
                        const uint4 q = lds128(sq + ((2 * b + e) * MT + mt) * QP * 512 + (i < 2 ? 512 : 0) + lane * 16);
#pragma unroll
                        for (int t = 0; t < GT; t++) mma16(p[t], q, e ? kw[t].z : kw[t].x, e ? kw[t].w : kw[t].y);
                    }
#pragma unroll
                    for (int t = 0; t < GT; t++) add4(s[mt][t], p[t]);
                }
            }
        } else {
#pragma unroll
            for (int b = 0; b < NB; b++) {
                uint32_t kh[GT][8], kl[GT][8];
#pragma unroll
                for (int t = 0; t < GT; t++)
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const uint4 w = lds128(base + (t * 8 + j) * C::RB + (((8 * b + 2 * c + u) ^ C::swk(j)) << 4));
                        cut_tf32(__uint_as_float(w.x), kh[t][4 * u], kl[t][4 * u]);
                        cut_tf32(__uint_as_float(w.y), kh[t][4 * u + 1], kl[t][4 * u + 1]);
                        cut_tf32(__uint_as_float(w.z), kh[t][4 * u + 2], kl[t][4 * u + 2]);
                        cut_tf32(__uint_as_float(w.w), kh[t][4 * u + 3], kl[t][4 * u + 3]);
                    }
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
                    float p[GT][4] = {};
#pragma unroll
                    for (int e = 0; e < 4; e++) {  // the small lo products first: what they are cut by is small
                        const uint4 qh = lds128(sq + ((4 * b + e) * MT + mt) * QP * 512 + lane * 16);
                        const uint4 ql = PACK ? qh : lds128(sq + ((4 * b + e) * MT + mt) * 1024 + 512 + lane * 16);
#pragma unroll
                        for (int t = 0; t < GT; t++) {
                            mma8(p[t], qh, kl[t][2 * e], kl[t][2 * e + 1]);
                            if (!PACK) mma8(p[t], ql, kh[t][2 * e], kh[t][2 * e + 1]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const uint4 qh = lds128(sq + ((4 * b + e) * MT + mt) * QP * 512 + lane * 16);
#pragma unroll
                        for (int t = 0; t < GT; t++) mma8(p[t], qh, kh[t][2 * e], kh[t][2 * e + 1]);
                    }
#pragma unroll
                    for (int t = 0; t < GT; t++) add4(s[mt][t], p[t]);
                }
            }
        }
        if (PACK)
#pragma unroll
            for (int t = 0; t < GT; t++) s[0][t][0] += s[0][t][2], s[0][t][1] += s[0][t][3];
        // ---- the slots of this walk of the stage, by the largest of their values' scales
        uint32_t dv[C::QUANT ? GT : 1][NB];
        again = false;
        if constexpr (C::QUANT) {
            __half2 most[GT], least = as_h2(0x7BFF7BFFu);  // by slot; of the slots that are not zeros
            auto find = [&](auto finite) {
#pragma unroll
                for (int t = 0; t < GT; t++) {
                    if (!decltype(finite)::value) load_scales<NB>(base + C::OVS + (t * 8 + 2 * c) * C::SB, dv[t]);
                    most[t] = as_h2(0u);
                    bool any = false;
#pragma unroll
                    for (int b = 0; b < NB; b++)
                        most[t] = __hmax2(most[t], __habs2(as_h2(decltype(finite)::value ? finite_h2(dv[t][b], any) : dv[t][b])));
                }
            };
            auto largest = [&]() {
                __half2 x = most[0];
#pragma unroll
                for (int t = 1; t < GT; t++) x = __hmax2(x, most[t]);
                return fmaxf(__low2float(x), __high2float(x));
            };
            find(std::false_type());
#pragma unroll
            for (int t = 0; t < GT; t++) least = __hmin2(least, __hfma2(__heq2(most[t], as_h2(0u)), as_h2(0x7BFF7BFFu), most[t]));
            const float small = fminf(__low2float(least), __high2float(least));
            if (__any_sync(0xffffffffu, todo != kAll || largest() > vlim || small < vlim * 0x1p-8f)) {
                find(std::true_type());  // of the finite scales (an infinite one stays one) that have not been walked
#pragma unroll
                for (int t = 0; t < GT; t++)
                    most[t] = as_h2(as_u(most[t]) & ((todo >> (2 * t) & 1 ? 0xFFFFu : 0u) | (todo >> (2 * t + 1) & 1 ? 0xFFFF0000u : 0u)));
                const float big = largest(), limit = big * 0x1p-7f;
                unsigned later = 0;
#pragma unroll
                for (int t = 0; t < GT; t++) {
                    const float x0 = __low2float(most[t]), x1 = __high2float(most[t]);
                    later |= (x0 != 0.f && x0 < limit ? 1u << (2 * t) : 0u) | (x1 != 0.f && x1 < limit ? 2u << (2 * t) : 0u);
                }
                const unsigned now = todo & ~later;
                todo = later;
                again = __any_sync(0xffffffffu, later != 0);
                if (now != kAll) {
#pragma unroll
                    for (int t = 0; t < GT; t++) {
                        const bool in0 = now >> (2 * t) & 1, in1 = now >> (2 * t + 1) & 1;
#pragma unroll
                        for (int b = 0; b < NB; b++) dv[t][b] &= (in0 ? 0xFFFFu : 0u) | (in1 ? 0xFFFF0000u : 0u);
#pragma unroll
                        for (int mt = 0; mt < MT; mt++)
#pragma unroll
                            for (int h = 0; h < NH; h++) {
                                if (!in0) s[mt][t][2 * h] = -CUDART_INF_F;
                                if (!in1) s[mt][t][2 * h + 1] = -CUDART_INF_F;
                            }
                    }
                }
                if (big > 0.f) {  // (2^-ev is an fp16 number)
                    const int e = min(max((int)(__float_as_uint(big) >> 23) - 127, -15), 14);
                    const float f = __uint_as_float((unsigned)(127 + e - (int)ev) << 23);  // (exactly: stages may take turns)
                    ev = (float)e;
                    vlim = __uint_as_float((unsigned)(e + 129) << 23);
#pragma unroll
                    for (int mt = 0; mt < MT; mt++)
#pragma unroll
                        for (int h = 0; h < NH; h++) l[mt][h] *= f;
                }
            }
        }
        // ---- mask and softmax
        float mx[MT][NH];
        bool move = false;
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
            for (int h = 0; h < NH; h++) {
                float x = -CUDART_INF_F;
#pragma unroll
                for (int t = 0; t < GT; t++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        float& v = s[mt][t][2 * h + i];
                        if (TYPE != AF_F32) v *= rowf[mt][h];
                        if (nodes && !(see[mt][h] >> (t * 8 + 2 * c + i) & 1)) v = -CUDART_INF_F;
                        x = fmaxf(x, v);
                    }
                mx[mt][h] = x;
                move |= x > m_ref[mt][h] + (C::QUANT ? fminf(ov[mt][h] - ev, 0.f) + kLazyT : kLazyT);
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int h = 0; h < NH; h++) {
                    float x = mx[mt][h], z = x + ev;
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    if (C::QUANT) {
                        z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 1));
                        z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 2));
                    }
                    const bool grow = C::QUANT && z > m_ref[mt][h] + ov[mt][h];
                    if (x > m_ref[mt][h] || grow) {
                        float d = x > m_ref[mt][h] ? m_ref[mt][h] - x : 0.f;
                        m_ref[mt][h] = fmaxf(m_ref[mt][h], x);
                        if (C::QUANT) {  // m + ov follows z, and stays (rounded up: p 2^ev grows no larger) when m moves alone
                            const float e = fmaxf(grow ? ceilf(z - m_ref[mt][h]) : ov[mt][h] + ceilf(d), -60.f);
                            d += ov[mt][h] - e;
                            ov[mt][h] = e;
                        }
                        const float f = ex2t(d);
                        l[mt][h] *= f;
#pragma unroll
                        for (int t = 0; t < NT; t++) {
                            o[mt][t][2 * h] *= f;
                            o[mt][t][2 * h + 1] *= f;
                            if (PACK) o[mt][t][2] *= f, o[mt][t][3] *= f;
                        }
                    }
                }
        }
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
            for (int h = 0; h < NH; h++) {
                const float mb = m_ref[mt][h] == -CUDART_INF_F ? 0.f : m_ref[mt][h] + (C::QUANT ? ov[mt][h] - ev - kBiasT : -kBiasT);
#pragma unroll
                for (int t = 0; t < GT; t++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float p = ex2t(s[mt][t][2 * h + i] - mb);
                        s[mt][t][2 * h + i] = p;
                        l[mt][h] += p;
                    }
            }
        // ---- output
        bool bad = false;  // non-finite values among the nodes' slots, taken out of the product
        if constexpr (C::QUANT) {
            const __half2 down = __float2half2_rn(__uint_as_float((256u << 23) - __float_as_uint(vlim)));
#pragma unroll
            for (int t = 0; t < GT; t++) {
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    if (nodes) dv[t][b] = finite_h2(dv[t][b], bad);
                    dv[t][b] = as_u(__hmul2(as_h2(dv[t][b]), down));
                }
            }
        }
        if constexpr (TYPE == AF_F32) {
            uint4 ph[GT][MT], pl[GT][MT];
#pragma unroll
            for (int t = 0; t < GT; t++)
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {  // slot 2c is k = c, slot 2c + 1 is k = c + 4
                    split_tf32(s[mt][t][0], ph[t][mt].x, PACK ? ph[t][mt].y : pl[t][mt].x);
                    split_tf32(s[mt][t][1], ph[t][mt].z, PACK ? ph[t][mt].w : pl[t][mt].z);
                    if (!PACK) {
                        split_tf32(s[mt][t][2], ph[t][mt].y, pl[t][mt].y);
                        split_tf32(s[mt][t][3], ph[t][mt].w, pl[t][mt].w);
                    }
                }
#pragma unroll
            for (int b = 0; b < NB; b++) {
                float sum[MT][4][4];  // of the stage
#pragma unroll
                for (int t = 0; t < GT; t++) {
                    const int k0 = t * 8 + 2 * c, k1 = k0 + 1;
                    const uint4 x = lds128(vb0 + k0 * C::RB + (((8 * b + j) ^ C::swv(k0)) << 4));
                    const uint4 y = lds128(vb0 + k1 * C::RB + (((8 * b + j) ^ C::swv(k1)) << 4));
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
                    uint32_t xh[4], xl[4], yh[4], yl[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        float fx = __uint_as_float(xs[i]), fy = __uint_as_float(ys[i]);
                        if (nodes) {
                            if (!(fabsf(fx) < CUDART_INF_F)) fx = 0.f, bad = true;
                            if (!(fabsf(fy) < CUDART_INF_F)) fy = 0.f, bad = true;
                        }
                        cut_tf32(fx, xh[i], xl[i]);
                        cut_tf32(fy, yh[i], yl[i]);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            if (t == 0)
                                mma8z(sum[mt][i], ph[t][mt], xl[i], yl[i]);
                            else
                                mma8(sum[mt][i], ph[t][mt], xl[i], yl[i]);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            if (!PACK) mma8(sum[mt][i], pl[t][mt], xh[i], yh[i]);
#pragma unroll
                        for (int i = 0; i < 4; i++) mma8(sum[mt][i], ph[t][mt], xh[i], yh[i]);
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int i = 0; i < 4; i++) add4(o[mt][4 * b + i], sum[mt][i]);
            }
        } else {
            constexpr int G16 = GT / 2;
            uint4 ph[G16][MT], pl[G16][MT];
#pragma unroll
            for (int g16 = 0; g16 < G16; g16++)
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
                    const float(&p0)[4] = s[mt][2 * g16], (&p1)[4] = s[mt][2 * g16 + 1];
                    split_h2(p0[0], p0[1], ph[g16][mt].x, PACK ? ph[g16][mt].y : pl[g16][mt].x);
                    split_h2(p1[0], p1[1], ph[g16][mt].z, PACK ? ph[g16][mt].w : pl[g16][mt].z);
                    if (!PACK) {
                        split_h2(p0[2], p0[3], ph[g16][mt].y, pl[g16][mt].y);
                        split_h2(p1[2], p1[3], ph[g16][mt].w, pl[g16][mt].w);
                    }
                }
            if constexpr (TYPE == AF_F16) {
                // lane: row lane & 15 of the 16 slots, chunk (lane >> 4) of the pair
                const int key = lane & 15;
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint4 v = ldsm4t(vb0 + key * C::RB + (((t + (lane >> 4)) ^ C::swv(key)) << 4));
                    if (nodes) {
                        v.x = finite_h2(v.x, bad), v.y = finite_h2(v.y, bad);
                        v.z = finite_h2(v.z, bad), v.w = finite_h2(v.w, bad);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; mt++) {
                        float x[4], y[4];
                        mma16z(x, PACK ? ph[0][mt] : pl[0][mt], v.x, v.y);
                        mma16z(y, PACK ? ph[0][mt] : pl[0][mt], v.z, v.w);
                        if (!PACK) {
                            mma16(x, ph[0][mt], v.x, v.y);
                            mma16(y, ph[0][mt], v.z, v.w);
                        }
                        add4(o[mt][t], x);
                        add4(o[mt][t + 1], y);
                    }
                }
            } else {
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    float sum[MT][4][4];  // of the stage
#pragma unroll
                    for (int g16 = 0; g16 < G16; g16++) {
                        const uint32_t vb = vb0 + g16 * 16 * C::RB;
                        uint32_t vw[4][2];
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int k0 = h * 8 + 2 * c, k1 = k0 + 1;
                            if (TYPE == AF_KV_Q8_0) {
                                const int byte = 32 * b + 4 * j;
                                const uint32_t w0 = lds32(vb + k0 * C::RB + ((((byte >> 4) ^ C::swv(k0)) << 4) | (byte & 15))) ^ 0x80808080u;
                                const uint32_t w1 = lds32(vb + k1 * C::RB + ((((byte >> 4) ^ C::swv(k1)) << 4) | (byte & 15))) ^ 0x80808080u;
                                const uint32_t x = __byte_perm(w0, w1, 0x5140), y = __byte_perm(w0, w1, 0x7362);
                                vw[0][h] = hsub2u(__byte_perm(x, 0x64646464u, 0x4140), 0x64806480u);
                                vw[1][h] = hsub2u(__byte_perm(x, 0x64646464u, 0x4342), 0x64806480u);
                                vw[2][h] = hsub2u(__byte_perm(y, 0x64646464u, 0x4140), 0x64806480u);
                                vw[3][h] = hsub2u(__byte_perm(y, 0x64646464u, 0x4342), 0x64806480u);
                            } else {
                                const uint32_t w = lds16(vb + k0 * C::RB + ((b ^ C::swv(k0)) << 4) + 2 * j) |
                                                   lds16(vb + k1 * C::RB + ((b ^ C::swv(k1)) << 4) + 2 * j) << 16;
#pragma unroll
                                for (int i = 0; i < 4; i++)
                                    vw[i][h] = hsub2u(((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u, 0x64086408u);
                            }
                        }
                        // p d in two parts: the fp16 product of p's high part, and what it lost plus p's low part's
                        const __half2 d0 = as_h2(dv[2 * g16][b]), d1 = as_h2(dv[2 * g16 + 1][b]);
#pragma unroll
                        for (int mt = 0; mt < MT; mt++) {
                            const uint4 qh = ph[g16][mt], ql = pl[g16][mt];
                            uint4 hi, lo;
                            auto times = [](uint32_t h, uint32_t l, __half2 d, uint32_t& hi, uint32_t& lo) {
                                const __half2 x = __hmul2_rn(as_h2(h), d);
                                hi = as_u(x);
                                lo = as_u(__hfma2(as_h2(l), d, __hfma2(as_h2(h), d, __hneg2(x))));
                            };
                            if (PACK) {
                                times(qh.x, qh.y, d0, hi.x, hi.y);
                                times(qh.z, qh.w, d1, hi.z, hi.w);
                            } else {
                                times(qh.x, ql.x, d0, hi.x, lo.x);
                                times(qh.y, ql.y, d0, hi.y, lo.y);
                                times(qh.z, ql.z, d1, hi.z, lo.z);
                                times(qh.w, ql.w, d1, hi.w, lo.w);
                            }
#pragma unroll
                            for (int t = 0; t < 4; t++)
                                if (g16 == 0)
                                    mma16z(sum[mt][t], PACK ? hi : lo, vw[t][0], vw[t][1]);
                                else
                                    mma16(sum[mt][t], PACK ? hi : lo, vw[t][0], vw[t][1]);
#pragma unroll
                            for (int t = 0; t < 4; t++)
                                if (!PACK) mma16(sum[mt][t], hi, vw[t][0], vw[t][1]);
                        }
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; mt++)
#pragma unroll
                        for (int t = 0; t < 4; t++) add4(o[mt][4 * b + t], sum[mt][t]);
                }
            }
        }
        if (nodes && __any_sync(0xffffffffu, bad)) {
            // rare: add p v of the non-finite values to the rows that see the slot
#pragma unroll
            for (int t8 = 0; t8 < GT; t8++)
#pragma unroll 1
                for (int k = 0; k < 8; k++) {
                    const int src = (lane & ~3) | (k >> 1), key = t8 * 8 + k;
#pragma unroll
                    for (int mt = 0; mt < MT; mt++)
#pragma unroll
                        for (int h = 0; h < NH; h++) {
                            const float p = __shfl_sync(0xffffffffu, (k & 1) ? s[mt][t8][2 * h + 1] : s[mt][t8][2 * h], src);
                            if (!(see[mt][h] >> key & 1)) continue;
#pragma unroll
                            for (int t = 0; t < NT; t++)
#pragma unroll
                                for (int i = 0; i < 2; i++) {
                                    const float v = stage_value<TYPE, D, MT_>(base, key, C::odim(t, 2 * c + i));
                                    if (!(fabsf(v) < CUDART_INF_F)) o[mt][t][2 * h + i] += p * v;
                                }
                        }
                }
        }
        if (!again) {
            todo = kAll;
            st += NW;
            slot = slot + 1 == C::NST ? 0 : slot + 1;
        }
    }
    cp_wait<0>();
    __syncthreads();

    if (PACK)
#pragma unroll
        for (int t = 0; t < NT; t++) o[0][t][0] += o[0][t][2], o[0][t][1] += o[0][t][3];
    // ---- join the warps: [warp][row][D] outputs, then [warp][row] (m, l)
    float* so = reinterpret_cast<float*>(smem + tree_q_bytes<TYPE, D, MT_>());
    float2* sml = reinterpret_cast<float2*>(so + NW * ROWS * C::DP);
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int h = 0; h < NH; h++) {
            const int r = mt * 16 + h * 8 + j;
            const float back = C::QUANT ? ex2t(ov[mt][h]) : 1.f;
            float x = C::QUANT ? l[mt][h] * ex2t(ov[mt][h] - ev) : l[mt][h];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if (c == 0) sml[warp * ROWS + r] = make_float2(m_ref[mt][h], x);
            float* dst = so + (warp * ROWS + r) * C::DP;
            if (TYPE == AF_F16) {
#pragma unroll
                for (int t = 0; t < NT; t++)
                    *reinterpret_cast<float2*>(dst + C::odim(t, 2 * c)) = make_float2(o[mt][t][2 * h], o[mt][t][2 * h + 1]);
            } else {  // tiles t..t+3 are neighbouring dims
#pragma unroll
                for (int t = 0; t < NT; t += 4)
#pragma unroll
                    for (int i = 0; i < 2; i++)
                        *reinterpret_cast<float4*>(dst + C::odim(t, 2 * c + i)) =
                            make_float4(o[mt][t][2 * h + i] * back, o[mt][t + 1][2 * h + i] * back,
                                        o[mt][t + 2][2 * h + i] * back, o[mt][t + 3][2 * h + i] * back);
            }
        }
    __syncthreads();
    float* part = a.ws;
    float2* part_ml = reinterpret_cast<float2*>(a.ws + (int64_t)splits * a.c.KVH * R * D);
    for (int i = threadIdx.x; i < ROWS * (D / 4); i += NW * 32) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        if (r0 + r >= R) break;
        float m = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < NW; w++) m = fmaxf(m, sml[w * ROWS + r].x);
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const float2 ml = sml[w * ROWS + r];
            if (ml.x == -CUDART_INF_F && ml.y == 0.f) continue;  // this warp saw nothing
            const float f = ex2t(ml.x - m);
            const float4 v = *reinterpret_cast<const float4*>(so + (w * ROWS + r) * C::DP + d);
            num.x += f * v.x, num.y += f * v.y, num.z += f * v.z, num.w += f * v.w;
            den += f * ml.y;
        }
        if (splits == 1) {
            const int node = (r0 + r) / G, head = g * G + (r0 + r) % G;
            const float inv = row_inverse(a, node, den);
            *reinterpret_cast<float4*>(a.out + (int64_t)node * a.ldo + (int64_t)head * D + d) =
                make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
        } else {
            const int64_t row = ((int64_t)split * a.c.KVH + g) * R + r0 + r;
            *reinterpret_cast<float4*>(part + row * D + d) = num;
            if (d == 0) part_ml[row] = make_float2(m, den);
        }
    }
}

// Joins the splits: W warps per row, each the parts s, s + W .. (eight loads in flight, issued with the maxima's), their
// sums in the warps' order.  One, two or four warps as there are parts: 25 nodes' 19 parts of 800 rows take 2.3 us less
// with four than with one warp that loads the maxima first, 64 nodes' 9 of 2048 rows 1.3 us less with two.  Blocks of
// 128 threads and 56 registers, so that one fits beside a block of the tcgen05 kernel and waits there.
template <int D, int W>
__global__ void __launch_bounds__(128, 9) tree_merge_kernel(TreeArgs a, int splits) {
    __shared__ float4 sums[4][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.H / a.c.KVH, R = a.n * G;
    const int rows = a.c.KVH * R, at = blockIdx.x * (4 / W) + warp / W, row = min(at, rows - 1), sub = warp % W;
    pdl_launch_dependents();
    pdl_wait();
    const float2* ml = reinterpret_cast<const float2*>(a.ws + (int64_t)splits * rows * D) + row;
    const int d = 4 * lane;
    const float* part = a.ws + (int64_t)row * D + (d < D ? d : 0);
    float2 x = make_float2(-CUDART_INF_F, 0.f);
    if (lane < splits) x = __ldcg(ml + (int64_t)lane * rows);
    float4 v[8];
    auto load = [&](int s) {  // this warp's next parts: s, s + W ..
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = s + i * W < splits ? __ldcg(reinterpret_cast<const float4*>(part + (int64_t)(s + i * W) * rows * D))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(sub);
    float m = x.x;
    for (int s = lane + 32; s < splits; s += 32) m = fmaxf(m, __ldcg(ml + (int64_t)s * rows).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
    for (int s0 = 0; s0 < splits; s0 += 32) {
        if (s0) {
            x = make_float2(-CUDART_INF_F, 0.f);
            if (s0 + lane < splits) x = __ldcg(ml + (int64_t)(s0 + lane) * rows);
        }
        const float w = x.x == -CUDART_INF_F && x.y == 0.f ? 0.f : ex2t(x.x - m);
        den += w * x.y;
        for (int s1 = 0; s1 < 32 && s0 + s1 < splits; s1 += 8 * W) {
            if (s0 + s1) load(s0 + s1 + sub);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float f = __shfl_sync(0xffffffffu, w, s1 + sub + i * W);
                num.x += f * v[i].x, num.y += f * v[i].y, num.z += f * v[i].z, num.w += f * v[i].w;
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (W > 1) {
        sums[warp][lane] = num;
        __syncthreads();
        if (sub) return;
#pragma unroll
        for (int i = 1; i < W; i++) {
            const float4 y = sums[warp + i][lane];
            num.x += y.x, num.y += y.y, num.z += y.z, num.w += y.w;
        }
    }
    if (d >= D || at >= rows) return;
    const int g = row / R, node = (row % R) / G, head = g * G + row % R % G;
    const float inv = row_inverse(a, node, den);
    *reinterpret_cast<float4*>(a.out + (int64_t)node * a.ldo + (int64_t)head * D + d) =
        make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
}

template <int D>
cudaError_t merge(const TreeArgs& a, int splits, cudaStream_t s) {
    const int rows = a.H * a.n;
    if (splits <= 8) return launch_chained(tree_merge_kernel<D, 1>, dim3((rows + 3) / 4), 128, 0, s, a, splits);
    if (splits <= 16) return launch_chained(tree_merge_kernel<D, 2>, dim3((rows + 1) / 2), 128, 0, s, a, splits);
    return launch_chained(tree_merge_kernel<D, 4>, dim3(rows), 128, 0, s, a, splits);
}

// The tcgen05 kernel, or this file's with one row tile of 8, 16 or 32 and so many splits that they fill the SMs, as long as
// every warp has a stage.
struct TreePlan {
    TreeTcPlan tc;
    int mt = 1, splits = 1;
};

TreePlan tree_plan(int H, int KVH, int D, int type, int past, int n) {
    TreePlan p;
    p.tc = tree_tc_plan(H, KVH, D, type, past, n);
    p.splits = p.tc.splits;
    if (p.splits) return p;
    const int R = n * (H / KVH);
    p.mt = R > 16 ? 2 : R > 8 ? 1 : 0;
    const int ks = tree_stage(type, p.mt), nw = tree_warps(type, D, p.mt);
    const int64_t tiles = KVH;  // (one row tile)
    const int stages = (past + n + ks - 1) / ks;
    int64_t s = num_sms() / tiles;
    s = std::min<int64_t>(s, (stages + nw - 1) / nw);
    p.splits = (int)std::max<int64_t>(1, s);
    return p;
}

template <int TYPE, int D, int MT>
cudaError_t go(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
    constexpr int smem = tree_smem<TYPE, D, MT>();
    auto k = attn_tree_kernel<TYPE, D, MT>;
    static SmemOptIn opt;
    cudaError_t e = opt((const void*)k, smem);
    if (e) return e;
    const int R = a.n * (a.H / a.c.KVH);
    constexpr int rows = TreeCfg<TYPE, D, MT>::ROWS;
    return launch_chained(k, dim3(p.splits, a.c.KVH, (R + rows - 1) / rows), TreeCfg<TYPE, D, MT>::NW * 32, smem, s, a, p.splits);
}

template <int TYPE>
cudaError_t go_type(const TreeArgs& a, cudaStream_t s) {
    const TreePlan p = tree_plan(a.H, a.c.KVH, a.c.D, TYPE, a.past, a.n);
    cudaError_t e;
    if (p.tc.splits)
        e = launch_attn_tree_tc(a, p.tc, s);
    else if (a.c.D == 64)
        e = p.mt == 0 ? go<TYPE, 64, 0>(a, p, s) : p.mt == 1 ? go<TYPE, 64, 1>(a, p, s) : go<TYPE, 64, 2>(a, p, s);
    else
        e = p.mt == 0 ? go<TYPE, 128, 0>(a, p, s) : p.mt == 1 ? go<TYPE, 128, 1>(a, p, s) : go<TYPE, 128, 2>(a, p, s);
    if (e || p.splits == 1) return e;
    return a.c.D == 64 ? merge<64>(a, p.splits, s) : merge<128>(a, p.splits, s);
}

}  // namespace

cudaError_t launch_tree_mask(const int* parent, int n, int pos0, unsigned* mask, int* pos, cudaStream_t s) {
    return launch_chained(tree_mask_kernel, dim3((n + 7) / 8), 256, 0, s, parent, n, pos0, mask, pos);
}

size_t attn_tree_ws_bytes(int H, int KVH, int D, int type, int past, int n) {
    const TreePlan p = tree_plan(H, KVH, D, type, past, n);
    if (p.splits == 1) return 0;
    return ((size_t)p.splits * n * H * (D + 2) * sizeof(float) + 255) & ~(size_t)255;
}

cudaError_t launch_attn_tree(const TreeArgs& a, cudaStream_t s) {
    switch (a.c.type) {
        case AF_F32: return go_type<AF_F32>(a, s);
        case AF_F16: return go_type<AF_F16>(a, s);
        case AF_KV_Q8_0: return go_type<AF_KV_Q8_0>(a, s);
        default: return go_type<AF_KV_Q4_0>(a, s);
    }
}

}  // namespace af

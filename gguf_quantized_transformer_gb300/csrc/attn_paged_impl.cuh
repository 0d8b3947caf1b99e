// Attention of single tokens over a paged cache: row r of the batch sees positions 0..pos_r of its request,
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(q . k_j / sqrt(D)),   k_j, v_j at slot table[seq][j / page] page + j % page.
// A row that sees no slot gives zeros; one whose scores are all -infinity has no softmax and gives NaN.
//
// Bound by the bytes of the cache: everything is arranged so that a warp does nothing but stream them.
//  - A work item is a row, a kv head and up to 4 NT heads of its group.  All items' stages of KS slots in a row are cut into
//    equal ranges, one per warp: no warp waits for another whatever the lengths are, one long request is spread over the
//    whole GPU and many short ones need no joining.  The ranges come from prefix sums of the rows' stages, which each
//    CTA forms from pos (at most kPagedMaxRows rows).
//  - K and V go from memory straight into the registers from which the matrix products take them: a stage's K is on its way
//    while the previous stage's softmax and output run, its V during the scores.  No shared memory and no barrier in the loop.
//  - Products have the slots as rows: S^T = K q^T with the columns (head 0 hi, head 0 lo, head 1 hi ..), q split into two
//    parts of 11 bits, so that a thread's two columns add up to one head's score; out^T = V^T p^T likewise, with p brought
//    into the operand's layout by 8x8 transposes (fp32: shuffles).  Four heads fill the 8 columns (a group of 8 takes two
//    column tiles).
//  - fp16: K and V are operands as they are.  Codes become fp16 integers: a key's scale multiplies its block's partial
//    score, a value's scale multiplies p in fp32 before p is split.
//  - fp32: K and V are cut into tf32 parts, three of the four products matter (the fourth comes with the columns).
//  - The reference of the softmax follows score + log2(the value's largest scale), so that what goes into the fp16 operand
//    (p times scale) stays below 2^14 and its low part above fp16's subnormal step whatever the scales; it moves only when
//    exceeded by more than 4.
//  - Tensor cores cut fp32 sums instead of rounding them: a stage's output and a block's score start from zero and are added
//    in fp32.
// Pieces of an item that several warps hold are joined through shared memory at the end of the CTA, those of several CTAs
// by paged_join_kernel, each in order: the bits do not change from call to call.
#pragma once
#include <math_constants.h>

#include "mma_sync.cuh"
#include "serve.cuh"
#include "tma.cuh"

namespace af {

constexpr float kLog2eP = 1.4426950408889634f;
constexpr float kLazyP = 4.f;   // powers of two by which the reference may be exceeded
constexpr float kBiasP = 10.f;  // p = 2^(s - m + kBiasP)

// What a CTA leaves for the join: its pieces 0 (an item that begins before it) and 1 (one that ends after it).
struct PagedPiece {
    int row, gi;    // gi = kv head * head tiles + head tile
    int used, ends;  // piece 0: whether the item ends in this CTA
};
constexpr int kPagedHeads = 8;  // heads of a piece at most
__host__ __device__ constexpr size_t paged_piece_floats(int D) { return (size_t)kPagedHeads * (D + 2); }
// ws: [ctas][2] pieces of paged_piece_floats (outputs [8][D], then [8] (m, l)), then [ctas][2] PagedPiece

template <int TYPE, int D, int NT>
struct PagedCfg {
    static constexpr bool QUANT = TYPE == AF_KV_Q8_0 || TYPE == AF_KV_Q4_0;
    static constexpr int NB = D / 32;
    static constexpr int RB = TYPE == AF_F32 ? 4 * D : TYPE == AF_F16 ? 2 * D : TYPE == AF_KV_Q8_0 ? D : D / 2;  // row bytes
    static constexpr int SB = QUANT ? 2 * NB : 0;
    static constexpr int SUB = QUANT ? 2 : 1;  // 16-slot tiles of a stage
    static constexpr int KS = 16 * SUB;
    static constexpr int KW = RB / 16;  // 32-bit words of K per thread, slot row and 16-slot tile (a quarter of a row)
    static constexpr int VW = RB / 32;  // of V (an eighth)
    static constexpr int STEPS = TYPE == AF_F32 ? D / 8 : D / 16;  // matrix steps along a head
    static constexpr int MT = D / 16;                              // row tiles of the output
    static constexpr int HEADS = 4 * NT;
    static constexpr int NW = TYPE == AF_F32 ? 8 : NT == 1 ? 12 : 8;  // warps
    static constexpr bool QSMEM = TYPE == AF_F32;  // q's operands in shared memory
    static constexpr int QBYTES = QSMEM ? NW * NT * STEPS * 32 * 8 : 0;
    static constexpr int PIECE = HEADS * (D + 2);  // floats of a warp's piece
    static constexpr int JOIN = NW * 2 * PIECE * 4;
    // first of the dims that lane c of a K row owns in block b (8 in a row)
    static __device__ __forceinline__ int kdim(int b, int c) {
        return TYPE == AF_KV_Q4_0 ? 32 * b + 8 * ((c & 1) * 2 + (c >> 1)) : 32 * b + 8 * c;
    }
};

// ---- loads through L2: what earlier kernels of the chain have written may be stale in L1
__device__ __forceinline__ void ldg16(const void* p, uint32_t* w) {
    const uint4 x = __ldcg(reinterpret_cast<const uint4*>(p));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
}
__device__ __forceinline__ void ldg8(const void* p, uint32_t* w) {
    const uint2 x = __ldcg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x, w[1] = x.y;
}
__device__ __forceinline__ uint32_t ldg4(const void* p) { return __ldcg(reinterpret_cast<const unsigned*>(p)); }

// 8x8 of 16 bits, transposed across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float lg2a(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// fp16 hi part in the low half, lo part in the high one
__device__ __forceinline__ uint32_t hi_lo(float x) {
    const float h = __uint_as_float(__float_as_uint(x) & 0xFFFFE000u);
    const __half2 r = __floats2half2_rn(h, x - h);
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ __half2 u_h2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t h2_u(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// The nibbles of both halves of a word as fp16 codes -8..7: place 0 of each half in r[0] and so on
__device__ __forceinline__ void codes4(uint32_t w, uint32_t (&r)[4]) {
    const __half2 f = __float2half2_rn(0.0625f), m72 = __float2half2_rn(-72.f);  // (1024 + 16 n) / 16 - 72
    const uint32_t z = w >> 8;
    r[0] = hsub2u((w & 0x000F000Fu) | 0x64006400u, 0x64086408u);
    r[1] = h2_u(__hfma2(u_h2((w & 0x00F000F0u) | 0x64006400u), f, m72));
    r[2] = hsub2u((z & 0x000F000Fu) | 0x64006400u, 0x64086408u);
    r[3] = h2_u(__hfma2(u_h2((z & 0x00F000F0u) | 0x64006400u), f, m72));
}

// A place in the order of all stages
struct PagedAt {
    int row, gi, st, nst;
};

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(PagedCfg<TYPE, D, NT>::NW * 32, 1) attn_paged_kernel(PagedArgs a) {
    using C = PagedCfg<TYPE, D, NT>;
    constexpr int NW = C::NW, KS = C::KS, SUB = C::SUB, NB = C::NB;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t sm_part[NW];
    __shared__ int4 sm_piece[NW][2];  // row, gi, used, ends
    uint32_t* const sq = reinterpret_cast<uint32_t*>(smem);
    float* const sjoin = reinterpret_cast<float*>(smem + C::QBYTES);
    int64_t* const first = reinterpret_cast<int64_t*>(smem + C::QBYTES + C::JOIN);  // [n + 1] stages of the rows before
    int2* const rows = reinterpret_cast<int2*>(first + a.n + 1);                     // [n] request, position
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, j = lane >> 2;
    const int KVH = a.c.KVH, G = a.H / KVH, HT = (G + C::HEADS - 1) / C::HEADS, GI = KVH * HT;

    pdl_wait();  // positions, tables, q and the cache are written by earlier kernels
    pdl_launch_dependents();  // (after the wait: the join may then read what they have written)
    // ---- stages of the rows and their prefix sums
    {
        const int per = (a.n + NW * 32 - 1) / (NW * 32), r0 = min(a.n, tid * per), r1 = min(a.n, r0 + per);
        const int64_t most = (int64_t)a.width * a.page;
        int64_t sum = 0;
        for (int r = r0; r < r1; r++) {
            const int who = a.seq ? __ldcg(a.seq + r) : r;
            int pos = __ldcg(a.pos + r);
            if (who < 0 || who >= a.n_seqs || pos < 0) pos = -1;
            if (pos >= most) pos = (int)(most - 1);
            rows[r] = make_int2(who, pos);
            first[r] = sum;
            sum += (pos + KS) / KS;
        }
        int64_t x = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sm_part[warp] = x;
        if (lane < 2) sm_piece[warp][lane] = make_int4(0, 0, 0, 0);
        __syncthreads();
        int64_t before = x - sum, total = 0;
#pragma unroll
        for (int w = 0; w < NW; w++) {
            if (w < warp) before += sm_part[w];
            total += sm_part[w];
        }
        for (int r = r0; r < r1; r++) first[r] += before;
        if (tid == 0) first[a.n] = total;
        __syncthreads();
    }
    const int64_t units = first[a.n] * GI, warps = (int64_t)gridDim.x * NW, me = (int64_t)blockIdx.x * NW + warp;
    // (units < 2^12 rows * 2^27 stages * 2^16 heads, so the product with the warps' number stays below 2^63 for units
    // below 2^51: above, the quotient comes first)
    auto cut = [&](int64_t w) { return units / warps * w + units % warps * w / warps; };
    int64_t u = cut(me);
    const int64_t u1 = cut(me + 1);

    // ---- rows that see nothing
    for (int r = blockIdx.x; r < a.n; r += gridDim.x)
        if (rows[r].y < 0)
            for (int d = tid; d < a.H * D / 4; d += NW * 32)
                *reinterpret_cast<float4*>(a.out + (int64_t)r * a.ldo + 4 * d) = make_float4(0.f, 0.f, 0.f, 0.f);

    if (u < u1) {
        PagedAt at;  // of the current stage
        {
            const int64_t x = u / GI;
            int lo = 0, hi = a.n;  // first[lo] <= x < first[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= x)
                    lo = mid;
                else
                    hi = mid;
            }
            at.row = lo;
            at.nst = (int)(first[lo + 1] - first[lo]);
            const int64_t y = u - first[lo] * GI;
            at.gi = (int)(y / at.nst);
            at.st = (int)(y - (int64_t)at.gi * at.nst);
        }
        auto advance = [&](PagedAt& p) {  // (behind the last stage: stays there)
            if (++p.st < p.nst) return;
            if (p.gi + 1 < GI) {
                p.st = 0;
                p.gi++;
                return;
            }
            int r = p.row + 1;
            while (r < a.n && first[r + 1] == first[r]) r++;
            if (r >= a.n) {
                p.st--;
                return;
            }
            p.row = r, p.gi = 0, p.st = 0, p.nst = (int)(first[r + 1] - first[r]);
        };
        // The table's entry for this lane's slot of a stage; -1 where it sees none
        auto look = [&](const PagedAt& p) -> int {
            const int2 w = rows[p.row];
            const int slot = p.st * KS + (KS == 32 ? lane : lane & 15);
            if (slot > w.y) return -1;
            const int pg = a.page_mul ? (int)(__umulhi((unsigned)slot, a.page_mul) >> a.page_shift) : slot;
            return __ldcg(a.table + (int64_t)w.x * a.width + pg);
        };
        // That entry as this lane's slot of the cache; -1 where it is hidden
        auto place = [&](const PagedAt& p, int pg) -> int {
            const int slot = p.st * KS + (KS == 32 ? lane : lane & 15);
            const int off = a.page_mul ? slot - (int)(__umulhi((unsigned)slot, a.page_mul) >> a.page_shift) * a.page : 0;
            return pg >= 0 && pg < a.n_pages ? pg * a.page + off : -1;
        };
        uint32_t kw[SUB][2][C::KW], vw[SUB][4][C::VW];
        uint2 ks[SUB][2], vs[SUB][2];
        // K of a stage: rows j and j + 8 of each 16, this lane's quarter of them.  Hidden slots read slot 0 of the pool.
        auto load_k = [&](int g, int phys) {
            const int64_t row0 = (int64_t)g * a.c.ctx;
#pragma unroll
            for (int s = 0; s < SUB; s++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int64_t row = row0 + max(__shfl_sync(0xffffffffu, phys, 16 * s + 8 * h + j), 0);
                    const uint8_t* p = (const uint8_t*)a.c.k + row * C::RB;
                    if constexpr (TYPE == AF_F32 || TYPE == AF_F16) {
#pragma unroll
                        for (int i = 0; i < C::KW / 4; i++) ldg16(p + (4 * i + c) * 16, &kw[s][h][4 * i]);
                    } else if constexpr (TYPE == AF_KV_Q8_0) {
#pragma unroll
                        for (int i = 0; i < NB; i++) ldg8(p + 32 * i + 8 * c, &kw[s][h][2 * i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < NB / 2; i++) ldg8(p + 32 * i + 8 * c, &kw[s][h][2 * i]);
                    }
                    if constexpr (C::QUANT) {
                        const uint8_t* q = (const uint8_t*)a.c.ks + row * C::SB;
                        if (NB == 4)
                            ks[s][h] = __ldcg(reinterpret_cast<const uint2*>(q));
                        else
                            ks[s][h].x = ldg4(q);
                    }
                }
        };
        // V: the four slots of each 16 that this lane has as an operand, its eighth of their rows
        auto load_v = [&](int g, int phys) {
            const int64_t row0 = (int64_t)g * a.c.ctx;
#pragma unroll
            for (int s = 0; s < SUB; s++) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int k = TYPE == AF_F32 ? c + 4 * i : 2 * c + (i & 1) + 8 * (i >> 1);
                    const int64_t row = row0 + max(__shfl_sync(0xffffffffu, phys, 16 * s + k), 0);
                    const uint8_t* p = (const uint8_t*)a.c.v + row * C::RB;
                    if constexpr (TYPE == AF_F32 || TYPE == AF_F16) {
#pragma unroll
                        for (int x = 0; x < C::VW / 4; x++) ldg16(p + (8 * x + j) * 16, &vw[s][i][4 * x]);
                    } else {
#pragma unroll
                        for (int x = 0; x < C::VW; x++) vw[s][i][x] = ldg4(p + 32 * x + 4 * j);
                    }
                }
                if constexpr (C::QUANT) {
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int64_t row = row0 + max(__shfl_sync(0xffffffffu, phys, 16 * s + 8 * h + j), 0);
                        const uint8_t* q = (const uint8_t*)a.c.vs + row * C::SB;
                        if (NB == 4)
                            vs[s][h] = __ldcg(reinterpret_cast<const uint2*>(q));
                        else
                            vs[s][h].x = ldg4(q);
                    }
                }
            }
        };

        // ---- the first stage is on its way, and the table's entries of the second
        PagedAt next = at;
        int phys = place(at, look(at));
        unsigned see = __ballot_sync(0xffffffffu, phys >= 0);
        load_k(at.gi / HT, phys);
        load_v(at.gi / HT, phys);
        advance(next);
        int entry = look(next);
        PagedAt after = next;

        uint32_t qf[C::QSMEM ? 1 : NT][C::QSMEM ? 1 : C::STEPS][2];  // q's operands
        float rowf[NT];
        float o[NT][C::MT][4], m_ref[NT], l[NT];
        bool seen = false, begun = true;  // begun: the piece begins with its item
        bool fresh = true;

        for (; u < u1; u++) {
            const int g = at.gi / HT, ht = at.gi - g * HT;
            // ---- where the next stage lies
            const int phys1 = place(next, entry);
            const unsigned see1 = __ballot_sync(0xffffffffu, phys1 >= 0);
            after = next;
            advance(after);
            entry = look(after);
            // ---- a new item: q's operands
            if (fresh) {
                fresh = false;
                begun = at.st == 0;
                seen = false;
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    m_ref[t] = -CUDART_INF_F;
                    l[t] = 0.f;
#pragma unroll
                    for (int i = 0; i < C::MT; i++) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
                    const int head = ht * C::HEADS + 4 * t + (j >> 1), part = j & 1;
                    float x[D / 4];  // this lane's quarter of the head
                    const float* q = a.q + (int64_t)at.row * a.ldq + (int64_t)(g * G + head) * D;
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        const int d = TYPE == AF_F32 ? 16 * i + 4 * c : C::kdim(i >> 1, c) + 4 * (i & 1);
                        const float4 v = head < G ? __ldcg(reinterpret_cast<const float4*>(q + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
                        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
                    }
                    const float sc = rsqrtf((float)D) * kLog2eP;
                    if constexpr (TYPE == AF_F32) {
#pragma unroll
                        for (int i = 0; i < D / 16; i++)
#pragma unroll
                            for (int e = 0; e < 4; e++) {  // dims 4c .. + 3 of 16: the two values of steps 2i and 2i + 1
                                uint32_t hi, lo;
                                split_tf32(x[4 * i + e] * sc, hi, lo);
                                sq[((warp * NT + t) * C::STEPS + 2 * i + (e >> 1)) * 64 + lane * 2 + (e & 1)] = part ? lo : hi;
                            }
                        rowf[t] = 1.f;
                    } else {
                        // a power of two brings the head's largest value to [2^12, 2^13)
                        float mx = 0.f;
#pragma unroll
                        for (int i = 0; i < D / 4; i++) x[i] *= sc, mx = fmaxf(mx, fabsf(x[i]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        int e = (int)(__float_as_uint(mx) >> 23) - 127 - 12;
                        e = e < -100 ? -100 : (e > 114 ? 114 : e);  // (0, subnormal; infinite: the row becomes NaN either way)
                        const float down = __uint_as_float((unsigned)(127 - e) << 23);
                        const float up = __uint_as_float((unsigned)(127 + e) << 23);
                        rowf[t] = __shfl_sync(0xffffffffu, up, 8 * c);  // of head c
#pragma unroll
                        for (int i = 0; i < D / 4; i++) {
                            x[i] *= down;
                            const uint32_t w = hi_lo(x[i]);
                            x[i] = __half2float(__ushort_as_half((unsigned short)(part ? w >> 16 : w)));  // this column's part
                        }
#pragma unroll
                        for (int b = 0; b < NB; b++) {
                            const float* y = x + 8 * b;
#pragma unroll
                            for (int i = 0; i < 4; i++)  // Q4_0: nibble i of a word's halves is dims i and i + 4
                                qf[t][2 * b + (i >> 1)][i & 1] = TYPE == AF_KV_Q4_0 ? h2_u(__floats2half2_rn(y[i], y[i + 4]))
                                                                                    : h2_u(__floats2half2_rn(y[2 * i], y[2 * i + 1]));
                        }
                    }
                }
                if (C::QSMEM) __syncwarp();
            }
            // ---- scores: s[t][16 s + ..]: this lane's slots j and j + 8 of each 16, head c of tile t
            float s[NT][SUB][2];
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int x = 0; x < SUB; x++) s[t][x][0] = s[t][x][1] = 0.f;
#pragma unroll
            for (int x = 0; x < SUB; x++) {
                if constexpr (TYPE == AF_F32) {
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        float p[NT][4] = {};
                        uint32_t lo[2][8];
#pragma unroll
                        for (int i = 0; i < 8; i++)
#pragma unroll
                            for (int h = 0; h < 2; h++) cut_tf32(__uint_as_float(kw[x][h][8 * b + i]), kw[x][h][8 * b + i], lo[h][i]);
#pragma unroll
                        for (int e = 0; e < 8; e++) {  // the small lo products first
                            const int i = 2 * (e & 3), step = 4 * b + (e & 3);
                            const uint32_t *k0 = e < 4 ? lo[0] : &kw[x][0][8 * b], *k1 = e < 4 ? lo[1] : &kw[x][1][8 * b];
#pragma unroll
                            for (int t = 0; t < NT; t++) {
                                const uint2 q = *reinterpret_cast<const uint2*>(sq + ((warp * NT + t) * C::STEPS + step) * 64 + lane * 2);
                                mma8(p[t], make_uint4(k0[i], k1[i], k0[i + 1], k1[i + 1]), q.x, q.y);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < NT; t++) s[t][x][0] += p[t][0] + p[t][1], s[t][x][1] += p[t][2] + p[t][3];
                    }
                } else {
                    uint32_t k4[2][NB];  // Q4_0: a word of each block
                    if constexpr (TYPE == AF_KV_Q4_0) {
#pragma unroll
                        for (int h = 0; h < 2; h++)
#pragma unroll
                            for (int i = 0; i < NB / 2; i++) {
                                // lanes c < 2 have 8 bytes of block 2i, the others of 2i + 1: one word of each is exchanged
                                const uint32_t w0 = kw[x][h][2 * i], w1 = kw[x][h][2 * i + 1];
                                const uint32_t got = __shfl_xor_sync(0xffffffffu, c < 2 ? w1 : w0, 2);
                                k4[h][2 * i] = c < 2 ? w0 : got;
                                k4[h][2 * i + 1] = c < 2 ? got : w1;
                            }
                    }
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        uint4 k[2];
                        if constexpr (TYPE == AF_F16) {
                            k[0] = make_uint4(kw[x][0][4 * b], kw[x][1][4 * b], kw[x][0][4 * b + 1], kw[x][1][4 * b + 1]);
                            k[1] = make_uint4(kw[x][0][4 * b + 2], kw[x][1][4 * b + 2], kw[x][0][4 * b + 3], kw[x][1][4 * b + 3]);
                        } else if constexpr (TYPE == AF_KV_Q8_0) {
                            uint32_t w[2][4];
#pragma unroll
                            for (int h = 0; h < 2; h++)
#pragma unroll
                                for (int i = 0; i < 2; i++) {
                                    const uint32_t y = kw[x][h][2 * b + i] ^ 0x80808080u;
                                    w[h][2 * i] = hsub2u(__byte_perm(y, 0x64646464u, 0x4140), 0x64806480u);
                                    w[h][2 * i + 1] = hsub2u(__byte_perm(y, 0x64646464u, 0x4342), 0x64806480u);
                                }
                            k[0] = make_uint4(w[0][0], w[1][0], w[0][1], w[1][1]);
                            k[1] = make_uint4(w[0][2], w[1][2], w[0][3], w[1][3]);
                        } else {
                            uint32_t w[2][4];
                            codes4(k4[0][b], w[0]);
                            codes4(k4[1][b], w[1]);
                            k[0] = make_uint4(w[0][0], w[1][0], w[0][1], w[1][1]);
                            k[1] = make_uint4(w[0][2], w[1][2], w[0][3], w[1][3]);
                        }
#pragma unroll
                        for (int t = 0; t < NT; t++) {
                            float p[4];
                            mma16z(p, k[0], qf[t][2 * b][0], qf[t][2 * b][1]);
                            mma16(p, k[1], qf[t][2 * b + 1][0], qf[t][2 * b + 1][1]);
                            const float s0 = p[0] + p[1], s1 = p[2] + p[3];
                            if constexpr (C::QUANT) {
                                const uint32_t d0 = b < 2 ? ks[x][0].x : ks[x][0].y, d1 = b < 2 ? ks[x][1].x : ks[x][1].y;
                                s[t][x][0] = fmaf(__half2float(b & 1 ? __high2half(u_h2(d0)) : __low2half(u_h2(d0))), s0, s[t][x][0]);
                                s[t][x][1] = fmaf(__half2float(b & 1 ? __high2half(u_h2(d1)) : __low2half(u_h2(d1))), s1, s[t][x][1]);
                            } else {
                                s[t][x][0] += s0;
                                s[t][x][1] += s1;
                            }
                        }
                    }
                }
            }
            // ---- K's registers take the next stage
            if (u + 1 < u1) load_k(next.gi / HT, phys1);
            // ---- softmax
            seen |= see != 0;
            if (see != 0xffffffffu) {  // hidden slots: no score, no value
#pragma unroll
                for (int x = 0; x < SUB; x++) {
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        if (!(see >> (16 * x + 8 * h + j) & 1)) {
#pragma unroll
                            for (int t = 0; t < NT; t++) s[t][x][h] = -CUDART_INF_F;
                            if (C::QUANT) vs[x][h] = make_uint2(0u, 0u);
                        }
                    if (!C::QUANT)
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int k = TYPE == AF_F32 ? c + 4 * i : 2 * c + (i & 1) + 8 * (i >> 1);
                            if (!(see >> (16 * x + k) & 1))
#pragma unroll
                                for (int w = 0; w < C::VW; w++) vw[x][i][w] = 0u;
                        }
                }
            }
            float big[SUB][2];  // log2 of the slots' largest value scales
            if constexpr (C::QUANT) {
#pragma unroll
                for (int x = 0; x < SUB; x++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        __half2 m = __habs2(u_h2(vs[x][h].x));
                        if (NB == 4) m = __hmax2(m, __habs2(u_h2(vs[x][h].y)));
                        big[x][h] = lg2a(fmaxf(fmaxf(__low2float(m), __high2float(m)), 0x1p-24f));
                    }
            }
            bool move = false;
            float mx[NT];
#pragma unroll
            for (int t = 0; t < NT; t++) {
                mx[t] = -CUDART_INF_F;
#pragma unroll
                for (int x = 0; x < SUB; x++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        if (TYPE != AF_F32) s[t][x][h] *= rowf[t];
                        mx[t] = fmaxf(mx[t], C::QUANT ? s[t][x][h] + big[x][h] : s[t][x][h]);
                    }
                move |= mx[t] > m_ref[t] + kLazyP;
            }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    float m = mx[t];
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    if (m > m_ref[t]) {
                        const float f = ex2t(m_ref[t] - m);
                        m_ref[t] = m;
                        l[t] *= f;
#pragma unroll
                        for (int i = 0; i < C::MT; i++)
#pragma unroll
                            for (int e = 0; e < 4; e++) o[t][i][e] *= f;
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < NT; t++) {
                const float mb = (m_ref[t] == -CUDART_INF_F ? 0.f : m_ref[t]) - kBiasP;
#pragma unroll
                for (int x = 0; x < SUB; x++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        s[t][x][h] = ex2t(s[t][x][h] - mb);
                        l[t] += s[t][x][h];
                    }
            }
            // ---- output
            if constexpr (TYPE == AF_F32) {
                uint32_t pb[NT][2][2];  // p of slots c + 8 u and c + 4 + 8 u for column j: its head's hi or lo part
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int v = 0; v < 2; v++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const float p = __shfl_sync(0xffffffffu, s[t][0][v], 4 * (c + 4 * h) + (j >> 1));
                            uint32_t hi, lo;
                            split_tf32(p, hi, lo);
                            pb[t][v][h] = j & 1 ? lo : hi;
                        }
#pragma unroll
                for (int i = 0; i < C::VW; i += 2) {  // the row tile of dims i and i + 1 of this lane's eighth
                    uint32_t lo[4][2], hi[4][2];
#pragma unroll
                    for (int k = 0; k < 4; k++)
#pragma unroll
                        for (int e = 0; e < 2; e++) cut_tf32(__uint_as_float(vw[0][k][i + e]), hi[k][e], lo[k][e]);
#pragma unroll
                    for (int t = 0; t < NT; t++) {
                        float sum[4];
                        mma8z(sum, make_uint4(lo[0][0], lo[0][1], lo[1][0], lo[1][1]), pb[t][0][0], pb[t][0][1]);
                        mma8(sum, make_uint4(lo[2][0], lo[2][1], lo[3][0], lo[3][1]), pb[t][1][0], pb[t][1][1]);
                        mma8(sum, make_uint4(hi[0][0], hi[0][1], hi[1][0], hi[1][1]), pb[t][0][0], pb[t][0][1]);
                        mma8(sum, make_uint4(hi[2][0], hi[2][1], hi[3][0], hi[3][1]), pb[t][1][0], pb[t][1][1]);
                        add4(o[t][i / 2], sum);
                    }
                }
            } else if constexpr (TYPE == AF_F16) {
                uint32_t pb[NT][2];
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int h = 0; h < 2; h++) pb[t][h] = transpose8(hi_lo(s[t][0][h]));
#pragma unroll
                for (int i = 0; i < C::VW; i++) {  // a word of the lane's eighth: two dims, one row tile
                    const uint4 v = make_uint4(__byte_perm(vw[0][0][i], vw[0][1][i], 0x5410), __byte_perm(vw[0][0][i], vw[0][1][i], 0x7632),
                                               __byte_perm(vw[0][2][i], vw[0][3][i], 0x5410), __byte_perm(vw[0][2][i], vw[0][3][i], 0x7632));
#pragma unroll
                    for (int t = 0; t < NT; t++) {
                        float sum[4];
                        mma16z(sum, v, pb[t][0], pb[t][1]);
                        add4(o[t][i], sum);
                    }
                }
            } else {
                uint32_t v4[SUB][2][NB];  // Q4_0: 16 bits of each of two slots, by pair of slots and block
                if constexpr (TYPE == AF_KV_Q4_0) {
#pragma unroll
                    for (int x = 0; x < SUB; x++)
#pragma unroll
                        for (int h = 0; h < 2; h++)
#pragma unroll
                            for (int i = 0; i < NB / 2; i++) {
                                // lanes j < 4 have 4 bytes of block 2i, the others of 2i + 1: half of them is exchanged
                                const uint32_t lo = __byte_perm(vw[x][2 * h][i], vw[x][2 * h + 1][i], 0x5410);
                                const uint32_t hi = __byte_perm(vw[x][2 * h][i], vw[x][2 * h + 1][i], 0x7632);
                                const uint32_t got = __shfl_xor_sync(0xffffffffu, j < 4 ? hi : lo, 16);
                                v4[x][h][2 * i] = j < 4 ? lo : got;
                                v4[x][h][2 * i + 1] = j < 4 ? got : hi;
                            }
                }
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    uint32_t pb[NT][SUB][2];
#pragma unroll
                    for (int x = 0; x < SUB; x++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const uint32_t w = b < 2 ? vs[x][h].x : vs[x][h].y;
                            const float d = __half2float(b & 1 ? __high2half(u_h2(w)) : __low2half(u_h2(w)));
#pragma unroll
                            for (int t = 0; t < NT; t++) pb[t][x][h] = transpose8(hi_lo(s[t][x][h] * d));
                        }
                    float sum[NT][2][4];
#pragma unroll
                    for (int x = 0; x < SUB; x++) {
                        uint32_t v[2][4];  // pair of slots, dim
#pragma unroll
                        for (int h = 0; h < 2; h++)
                            if constexpr (TYPE == AF_KV_Q8_0) {
                                const uint32_t w0 = vw[x][2 * h][b] ^ 0x80808080u, w1 = vw[x][2 * h + 1][b] ^ 0x80808080u;
                                const uint32_t y = __byte_perm(w0, w1, 0x5140), z = __byte_perm(w0, w1, 0x7362);
                                v[h][0] = hsub2u(__byte_perm(y, 0x64646464u, 0x4140), 0x64806480u);
                                v[h][1] = hsub2u(__byte_perm(y, 0x64646464u, 0x4342), 0x64806480u);
                                v[h][2] = hsub2u(__byte_perm(z, 0x64646464u, 0x4140), 0x64806480u);
                                v[h][3] = hsub2u(__byte_perm(z, 0x64646464u, 0x4342), 0x64806480u);
                            } else {
                                codes4(v4[x][h][b], v[h]);
                            }
#pragma unroll
                        for (int t = 0; t < NT; t++)
#pragma unroll
                            for (int i = 0; i < 2; i++) {
                                const uint4 w = make_uint4(v[0][2 * i], v[0][2 * i + 1], v[1][2 * i], v[1][2 * i + 1]);
                                if (x == 0)
                                    mma16z(sum[t][i], w, pb[t][x][0], pb[t][x][1]);
                                else
                                    mma16(sum[t][i], w, pb[t][x][0], pb[t][x][1]);
                            }
                    }
#pragma unroll
                    for (int t = 0; t < NT; t++)
#pragma unroll
                        for (int i = 0; i < 2; i++) add4(o[t][2 * b + i], sum[t][i]);
                }
            }
            // ---- V's registers take the next stage
            if (u + 1 < u1) load_v(next.gi / HT, phys1);

            // ---- the end of the item, or of this warp's range
            const bool ends = at.st + 1 == at.nst;
            if (ends || u + 1 == u1) {
                fresh = true;
                const bool done = begun && ends;
                const int slot = begun ? 1 : 0;
                float* piece = sjoin + (warp * 2 + slot) * C::PIECE;
                if (!done && lane == 0) sm_piece[warp][slot] = make_int4(at.row, at.gi, 1, ends);
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    float x = l[t];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    if (x == 0.f && seen) x = -0.f;  // (a sum that saw slots: +0 means none were)
                    const int hh = 4 * t + c, head = ht * C::HEADS + hh;
                    const float inv = !done ? 1.f : x != 0.f ? 1.f / x : seen ? CUDART_NAN_F : 0.f;
                    float* dst = done ? a.out + (int64_t)at.row * a.ldo + (int64_t)(g * G + head) * D : piece + hh * D;
                    if (!done && j == 0) reinterpret_cast<float2*>(piece + C::HEADS * D)[hh] = make_float2(m_ref[t], x);
                    if (!done || head < G) {
                        // row tile i: dims (j) and (j + 8) of its output are neighbours, i and i + 1 make four
#pragma unroll
                        for (int i = 0; i < C::MT; i += 2) {
                            const int d = TYPE == AF_F16   ? 64 * (i >> 2) + 8 * j + 2 * (i & 3)
                                          : TYPE == AF_F32 ? 32 * (i >> 1) + 4 * j
                                          : TYPE == AF_KV_Q8_0
                                              ? 16 * i + 4 * j
                                              : 16 * i + (j < 4 ? 8 * j : 8 * (j - 4) + 4);
                            *reinterpret_cast<float4*>(dst + d) =
                                make_float4((o[t][i][0] + o[t][i][1]) * inv, (o[t][i][2] + o[t][i][3]) * inv,
                                            (o[t][i + 1][0] + o[t][i + 1][1]) * inv, (o[t][i + 1][2] + o[t][i + 1][3]) * inv);
                        }
                    }
                }
            }
            at = next;
            next = after;
            see = see1;
        }
    }

    // ---- join: chains of pieces in the order of the warps; a warp takes every NW-th head of all chains
    __syncthreads();
    PagedPiece* const info = reinterpret_cast<PagedPiece*>(a.ws + (size_t)gridDim.x * 2 * paged_piece_floats(D));
    int job = 0;
    bool head0 = false, tail1 = false;  // the CTA's own pieces
    int covered = -1;                    // the last warp whose piece 0 belongs to a chain
    for (int w = 0; w < NW; w++)
        for (int slot = 0; slot < 2; slot++) {
            const int4 p = sm_piece[w][slot];
            if (!p.z || (slot == 0 && w <= covered)) continue;
            // where the chain ends
            bool ends = p.w;
            int last = w;
            for (int x = w + 1; x < NW && !ends; x++) {
                const int4 y = sm_piece[x][0];
                if (y.z) last = x, ends = y.w;
            }
            covered = last;
            const bool out = slot == 1 && ends;
            if (!out && tid == 0) info[blockIdx.x * 2 + slot] = PagedPiece{p.x, p.y, 1, ends};
            if (!out) (slot ? tail1 : head0) = true;
            const int g = p.y / HT, ht = p.y - g * HT;
            for (int hh = 0; hh < C::HEADS; hh++, job++) {
                if (job % NW != warp || ht * C::HEADS + hh >= G) continue;
                auto piece = [&](int x) { return sjoin + (x * 2 + (x == w ? slot : 0)) * C::PIECE; };
                auto stat = [&](int x) { return reinterpret_cast<const float2*>(piece(x) + C::HEADS * D)[hh]; };
                float m = -CUDART_INF_F;
                for (int x = w; x <= last; x++)
                    if (x == w || sm_piece[x][0].z) m = fmaxf(m, stat(x).x);
                float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
                float den = 0.f;
                bool saw = false;
                for (int x = w; x <= last; x++) {
                    if (x != w && !sm_piece[x][0].z) continue;
                    const float2 ml = stat(x);
                    saw |= __float_as_uint(ml.y) != 0;
                    if (ml.x == -CUDART_INF_F && ml.y == 0.f) continue;
                    const float f = ex2t(ml.x - m);
                    den += f * ml.y;
                    if (4 * lane < D) {
                        const float4 v = *reinterpret_cast<const float4*>(piece(x) + hh * D + 4 * lane);
                        num.x += f * v.x, num.y += f * v.y, num.z += f * v.z, num.w += f * v.w;
                    }
                }
                if (out) {
                    const float inv = den != 0.f ? 1.f / den : saw ? CUDART_NAN_F : 0.f;
                    if (4 * lane < D)
                        *reinterpret_cast<float4*>(a.out + (int64_t)p.x * a.ldo + (int64_t)(g * G + ht * C::HEADS + hh) * D + 4 * lane) =
                            make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
                } else {
                    float* dst = a.ws + (size_t)(blockIdx.x * 2 + slot) * paged_piece_floats(D);
                    if (4 * lane < D) *reinterpret_cast<float4*>(dst + hh * D + 4 * lane) = num;
                    if (den == 0.f && saw) den = -0.f;
                    if (lane == 0) reinterpret_cast<float2*>(dst + kPagedHeads * D)[hh] = make_float2(m, den);
                }
            }
        }
    if (tid == 0) {
        if (!head0) info[blockIdx.x * 2] = PagedPiece{0, 0, 0, 0};
        if (!tail1) info[blockIdx.x * 2 + 1] = PagedPiece{0, 0, 0, 0};
    }
}

// One translation unit per cache type.
template <int TYPE>
cudaError_t launch_attn_paged_type(const PagedArgs& a, int ctas, cudaStream_t s);

template <int TYPE, int D, int NT>
cudaError_t paged_go(const PagedArgs& a, int ctas, cudaStream_t s) {
    using C = PagedCfg<TYPE, D, NT>;
    constexpr int fixed = C::QBYTES + C::JOIN;
    static_assert(fixed + (kPagedMaxRows + 1) * 8 + kPagedMaxRows * 8 <= 220 * 1024, "shared memory");
    auto k = attn_paged_kernel<TYPE, D, NT>;
    static SmemOptIn opt;
    cudaError_t e = opt((const void*)k, fixed + (kPagedMaxRows + 1) * 8 + kPagedMaxRows * 8);
    if (e) return e;
    return launch_chained(k, dim3(ctas), C::NW * 32, fixed + (a.n + 1) * 8 + a.n * 8, s, a);
}

#define AF_PAGED_INSTANTIATE(TYPE)                                                                    \
    template <>                                                                                       \
    cudaError_t launch_attn_paged_type<TYPE>(const PagedArgs& a, int ctas, cudaStream_t s) {          \
        const int G = a.H / a.c.KVH;                                                                  \
        if (a.c.D == 64) return G > 4 ? paged_go<TYPE, 64, 2>(a, ctas, s) : paged_go<TYPE, 64, 1>(a, ctas, s); \
        return G > 4 ? paged_go<TYPE, 128, 2>(a, ctas, s) : paged_go<TYPE, 128, 1>(a, ctas, s);       \
    }

}  // namespace af

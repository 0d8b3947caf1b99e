// Attention of single tokens over a paged cache: row r of the batch sees positions 0..pos_r of its request,
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(q . k_j / sqrt(D)),   k_j, v_j at slot table[seq][j / page] page + j % page.
// A row that sees no slot gives zeros; one whose scores are all -infinity has no softmax and gives NaN.
//
// Bound by the bytes of the cache (of the measured copy rate, for long batches with groups of 4: fp32 0.92 to 1.0, fp16 0.93 to
// 0.97, Q8_0 with heads of 128 0.84 to 0.90), for few slots by its chain of dependent loads.  Q4_0 (0.51), heads of 64 with codes
// (Q8_0 0.70, Q4_0 0.37) and fp32 with groups of 8 (0.78, the tf32 rate of mma.sync) are bound in the SM: for Q4_0 issue is 65%
// full and the ALU pipe 59%, next to nothing waits for memory, and a scheduler's three warps mostly wait for their own last
// results.  How it is laid out:
//  - A work item is a row, a kv head and up to 4 NT heads of its group.  (A group above 8 is several items, each of which copies and
//    unpacks K and V: 16 rows of 8000 fp16 slots 51 us with groups of 8, 88 with 16, 162 with 32.  A group of 5 costs what one of
//    8 does.  New tokens of one request are items of their own too: 8 requests with 8 each over 4096 slots take 119 us, with one
//    each 29.)  All items' stages of KS slots in a row are cut into
//    equal ranges, one per warp: no warp waits for another whatever the lengths are, one long request is spread over the
//    whole GPU and many short ones need little joining.  The ranges come from prefix sums of the rows' stages, which each
//    CTA forms from pos (at most kPagedMaxRows rows).
//  - A warp streams its range through a ring of its own, two stages of K and V by 16-byte asynchronous copies, K's part
//    refilled while the softmax runs and V's during the next scores; no barrier but __syncwarp in the loop.  (Loads straight
//    into operand registers, the first design, took 236 us where this takes 173: 64 fp16 requests of up to 8192 x 128.)
//    A lane holds two entries of the table's row, so that 64 pages' addresses are shuffles; 16 neighbouring slots
//    (pages of a multiple of 16) are copied from one address.
//  - Products have the slots as rows: S^T = K q^T with the columns (head 0 hi, head 0 lo, head 1 hi ..), q split into two
//    parts of 11 bits, so that a thread's two columns add up to one head's score; out^T = V^T p^T likewise, with p brought
//    into the operand's layout by 8x8 transposes (fp32: shuffles).  Four heads fill the 8 columns (a group of 8 takes two
//    column tiles).
//  - fp16: K and V are operands as they are.  Codes become fp16 integers: a key's scale multiplies its block's partial
//    score, a value's scale multiplies p in fp32 before p is split.  (Codes with their offset left in, which saves a third of
//    the unpacking, lose three bits of a score: 1.3e-6 of the result's norm in place of 4e-7.)
//  - fp32: K and V are cut into tf32 parts, three of the four products matter (the fourth comes with the columns).
//  - The reference of the softmax follows score + log2(the value's largest scale), so that what goes into the fp16 operand
//    (p times scale) stays below 2^14 and its low part above fp16's subnormal step whatever the scales; it moves only when
//    exceeded by more than 4.
//  - Tensor cores cut fp32 sums instead of rounding them: a stage's output and a block's score start from zero and are added
//    in fp32.
// Pieces of an item that several warps hold are joined through shared memory at the end of the CTA, those of several CTAs
// by the last of them to leave its own (a second kernel took 4 to 5 us more), each in order: the bits do not change from
// call to call.
#pragma once
#include <math_constants.h>

#include <type_traits>

#include "mma_sync.cuh"
#include "serve.cuh"
#include "tma.cuh"

namespace af {

constexpr float kLog2eP = 1.4426950408889634f;
constexpr float kLazyP = 4.f;   // powers of two by which the reference may be exceeded
constexpr float kBiasP = 10.f;  // p = 2^(s - m + kBiasP)

constexpr int kPagedKept = 512;  // rows whose request and position a CTA keeps
constexpr int kPagedHeads = 8;   // heads of a piece at most
// The workspace: a counter per CTA (of the CTAs that have left their part of the item that begins in it); each CTA's pieces
// 0 (of an item that begins before it) and 1 (of one that goes on after it), outputs [8][D] and then [8] (m, l); the pieces
// of warps that go on after them: 16 warps of 4 heads or 8 of 8.
__host__ __device__ constexpr size_t paged_piece_floats(int D) { return (size_t)kPagedHeads * (D + 2); }
__host__ __device__ constexpr size_t paged_pieces(int ctas) { return ((size_t)ctas * 2 + 63) / 64 * 64; }
__host__ __device__ constexpr size_t paged_far(int ctas, int D) { return paged_pieces(ctas) + (size_t)ctas * 2 * paged_piece_floats(D); }
__host__ __device__ constexpr size_t paged_ws_floats(int ctas, int D) {
    return paged_far(ctas, D) + (size_t)ctas * 8 * paged_piece_floats(D);
}

// Warps of a CTA (one to an SM): as many as their registers and rings allow, but for fp16 rows of 128 and fp32 ones, where more
// only lengthen the joins (fp16, one token over 30720 slots 28.6 us with 8 warps, 29.7 with 12; fp32 rows of 64 312 and 329
// with 8 and 12; fp16 rows of 64 190 and 168 with 8 and 12, Q8_0 ones 133 and 121 with 12 and 16).
__host__ __device__ constexpr int paged_warps(int type, int D, int nt) {
    return type == AF_F32 ? (D == 128 ? 6 : 8) : nt == 2 ? 8 : D == 64 ? (type == AF_F16 ? 12 : 16) : (type == AF_F16 ? 8 : 12);
}

template <int TYPE, int D, int NT>
struct PagedCfg {
    static constexpr bool QUANT = TYPE == AF_KV_Q8_0 || TYPE == AF_KV_Q4_0;
    static constexpr int NB = D / 32;
    static constexpr int RB = TYPE == AF_F32 ? 4 * D : TYPE == AF_F16 ? 2 * D : TYPE == AF_KV_Q8_0 ? D : D / 2;  // row bytes
    static constexpr int SB = QUANT ? 2 * NB : 0;  // scale bytes of a row
    static constexpr int SUB = QUANT ? 2 : 1;      // 16-slot tiles of a stage
    static constexpr int KS = 16 * SUB;
    static constexpr int STEPS = TYPE == AF_F32 ? D / 8 : D / 16;  // matrix steps along a head
    static constexpr int MT = D / 16;                              // row tiles of the output
    static constexpr int HEADS = 4 * NT;
    static constexpr int NW = paged_warps(TYPE, D, NT);
    // a stage: K rows, V rows, and the 16 bytes around each slot's K and V scales
    static constexpr int OV = KS * RB, OKS = 2 * KS * RB, OVS = OKS + (QUANT ? 16 * KS : 0);
    static constexpr int STAGE = OVS + (QUANT ? 16 * KS : 0);
    static constexpr int NST = 2;  // stages of a warp's ring (three, which no longer fit, were 1 to 2% slower)
    static constexpr int PIECE = HEADS * (D + 2);  // floats of a warp's piece
    static_assert(PIECE * 4 <= NST * STAGE, "a piece fits the ring");
    static constexpr int RING = NW * NST * STAGE, ROWS = (kPagedMaxRows + 1) * 4, STATIC = NW * (32 + 16 * NST + 8) + 256;
    static constexpr bool NEAR = RING + ROWS + STATIC + NW * PIECE * 4 <= 227 * 1024;  // pieces of warps that go on fit beside it
    static constexpr int FIXED = RING + (NEAR ? NW * PIECE * 4 : 0);
    static_assert(FIXED + ROWS + STATIC <= 227 * 1024, "shared memory");
    // 16-byte chunk permutations within 128 bytes, by row, so that the reads of a warp meet all banks (codes: eight rows in a
    // row)
    static __device__ __forceinline__ constexpr int swk(int r) {
        if (!QUANT) return (r & 1) << 2;
        return RB == 128 ? r & 7 : RB == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
    }
    static __device__ __forceinline__ constexpr int swv(int r) {
        if (TYPE == AF_F32) return (r & 3) << 1;
        if (TYPE == AF_F16) return ((r >> 1) & 3) << 1;
        return swk(r);
    }
    // where byte `at` of row r lies
    static __device__ __forceinline__ int kbyte(int r, int at) { return (r * RB + at) ^ (swk(r) << 4); }
    static __device__ __forceinline__ int vbyte(int r, int at) { return OV + ((r * RB + at) ^ (swv(r) << 4)); }
    // Slot of K's row r of 16, and of row j of half h of a matrix operand: transposed bytes give a lane c four slots in a row of V,
    // and its operands' pairs are what takes the fewest instructions: (4c, 4c + 1) and (4c + 2, 4c + 3), of nibbles (4c, 4c + 2)
    // and (4c + 1, 4c + 3).
    static __device__ __forceinline__ constexpr int kslot(int r) {
        return QUANT ? 4 * ((r & 7) >> 1) + (r & 1) + 2 * (r >> 3) : r;
    }
    static __device__ __forceinline__ int slot(int h, int j) { return kslot(8 * h + j); }
};

// 16 bytes from global to shared memory through L2 (what earlier kernels of the chain have written may be stale in L1), of
// which the first `bytes` are read and the others zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void shared128(uint32_t a, uint32_t* w) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
}
__device__ __forceinline__ void shared64(uint32_t a, uint32_t* w) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
}
__device__ __forceinline__ uint32_t shared32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t shared16(uint32_t a) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}

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

// Four 8x8 matrices of 16 bits: lane (j, c) gets the 4 bytes at 4c of each one's row j.  Lanes 8i.. give matrix i's rows.
__device__ __forceinline__ void rows4(uint32_t a, uint32_t* w) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a));
}
// Two 16x16 matrices of bytes, transposed: lane (j, c) gets columns j and j + 8 of each, of rows 4c .. 4c + 3.  Lanes 16i.. give
// matrix i's rows.
__device__ __forceinline__ void columns4(uint32_t a, uint32_t* w) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a));
}
// Four signed bytes as fp16 pairs
__device__ __forceinline__ void codes2(uint32_t w, uint32_t& a, uint32_t& b) {
    w ^= 0x80808080u;
    a = hsub2u(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u);
    b = hsub2u(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u);
}
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
    constexpr int NW = C::NW, KS = C::KS, SUB = C::SUB, NB = C::NB, NST = C::NST;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t sm_part[NW];  // (32 or 64 bits)
    __shared__ int4 sm_piece[NW][2];   // row, gi, used (1: in the ring, 2: in the workspace), ends
    __shared__ uint4 sm_head[NW][NST];  // of a stage in flight: the slots that are seen, and two bits of where their scales lie
    int2* const rows = reinterpret_cast<int2*>(smem + C::FIXED);  // [n] request and position, for up to kPagedKept rows
    int* const first = reinterpret_cast<int*>(rows + (a.n <= kPagedKept ? a.n : 0));  // [n + 1] stages before each row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, j = lane >> 2;
    const int KVH = a.c.KVH, G = a.H / KVH, HT = (G + C::HEADS - 1) / C::HEADS, GI = KVH * HT;
    const uint32_t ring = smem_u32(smem) + warp * NST * C::STAGE;
    float* const my_piece = reinterpret_cast<float*>(smem + warp * NST * C::STAGE);
    // pieces of warps whose ring goes on
    float* const far = C::NEAR ? reinterpret_cast<float*>(smem + C::RING) : a.ws + paged_far(gridDim.x, D) + (size_t)blockIdx.x * NW * C::PIECE;

    pdl_wait();  // positions, tables, q and the cache are written by earlier kernels
    // request and last position of a row; -1: it sees nothing
    auto row_of = [&](int r) {
        const int who = a.seq ? __ldcg(a.seq + r) : r;
        int pos = __ldcg(a.pos + r);
        if (who < 0 || who >= a.n_seqs || pos < 0) pos = -1;
        return make_int2(who, min(pos, a.width * a.page - 1));
    };
    const bool kept = a.n <= kPagedKept;
    auto row_at = [&](int r) { return kept ? rows[r] : row_of(r); };
    // ---- stages of the rows and their prefix sums, counted from the stage with which this CTA begins; each warp's range.
    // (I: 32 bits where they hold all stages of all items)
    const int per = (a.n + NW * 32 - 1) / (NW * 32), r0 = min(a.n, tid * per), r1 = min(a.n, r0 + per);
    int64_t u, u1, begin_unit, units_each, units_rest;
    auto plan = [&](auto zero, int64_t* parts) {
        using I = decltype(zero);
        I* const part = reinterpret_cast<I*>(parts);
        I sum = 0;
#pragma unroll 1
        for (int r = r0; r < r1; r++) {
            const int2 w = row_of(r);
            if (kept) rows[r] = w;
            first[r] = (w.y + KS) / KS;
            sum += first[r];
        }
        I x = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const I y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) part[warp] = x;
        if (lane < 2) sm_piece[warp][lane] = make_int4(0, 0, 0, 0);
        __syncthreads();
        x -= sum;
        I total = 0;
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const I y = part[w];
            if (w < warp) x += y;
            total += y;
        }
        // the first `rest` warps have a stage more than the others; a warp has at least 32 slots, so that short items of a
        // small call need no joining (chosen by calls with groups of 4 and 8)
        const I units = total * GI, warps = gridDim.x * NW, least = 32 / KS;
        I each = units / warps, rest = units - each * warps;
        if (each < least) each = least, rest = 0;
        auto cut = [&](I w) { return min(each * w + min(w, rest), units); };
        const I me = blockIdx.x * NW, begin = cut(me) / GI;
        begin_unit = (int64_t)begin * GI, units_each = each, units_rest = rest;
        u = cut(me + warp) - begin * GI;
        u1 = cut(me + warp + 1) - begin * GI;
        // (2048 rows of at most 2^27 stages over 152 CTAs: a CTA's own fit 31 bits)
        auto from_here = [&](I at) { return (int)max(min((int64_t)at - begin, (int64_t)INT32_MAX), (int64_t)INT32_MIN); };
#pragma unroll 1
        for (int r = r0; r < r1; r++) {
            const int stages = first[r];
            first[r] = from_here(x);
            x += stages;
        }
        if (tid == 0) first[a.n] = from_here(total);
        __syncthreads();
    };
    if (a.wide)
        plan((int64_t)0, sm_part);
    else
        plan((int)0, sm_part);
    for (int r = blockIdx.x; r < a.n; r += gridDim.x)  // rows that see nothing
        if (row_at(r).y < 0)
            for (int d = tid; d < a.H * D / 4; d += NW * 32)
                *reinterpret_cast<float4*>(a.out + (int64_t)r * a.ldo + 4 * d) = make_float4(0.f, 0.f, 0.f, 0.f);
    unsigned long long* const counters = reinterpret_cast<unsigned long long*>(a.ws);
    auto cta_of = [&](int64_t unit) {
        const int64_t more = units_rest * (units_each + 1);
        if (!a.wide)
            return (int)((unit < more ? (unsigned)unit / (unsigned)(units_each + 1)
                                      : (unsigned)units_rest + (unsigned)(unit - more) / max((unsigned)units_each, 1u)) / NW);
        return (int)((unit < more ? unit / (units_each + 1) : units_rest + (unit - more) / max(units_each, (int64_t)1)) / NW);
    };
    const bool any = u < u1;
    if (any) {
        PagedAt at;  // the stage that is computed
        {
            const int x = u <= INT32_MAX ? (int)u / GI : (int)(u / GI);
            int lo = 0, hi = a.n;  // first[lo] <= x < first[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= x)
                    lo = mid;
                else
                    hi = mid;
            }
            at.row = lo;
            at.nst = first[lo + 1] - first[lo];
            const int64_t y = u - (int64_t)first[lo] * GI;
            at.gi = y <= INT32_MAX ? (int)y / at.nst : (int)(y / at.nst);
            at.st = (int)(y - (int64_t)at.gi * at.nst);
        }
        auto next_row = [&](int r) {
            for (r++; r < a.n && first[r + 1] == first[r]; r++) {
            }
            return r;
        };
        auto page_of = [&](int slot) { return a.page_mul ? (int)(__umulhi((unsigned)slot, a.page_mul) >> a.page_shift) : slot; };
        int left = (int)min(u1 - u, (int64_t)INT32_MAX);  // stages of this warp to compute, and to fetch (more are as good)
        int fetch = left;
        // ---- the stage that is fetched next and its row; 64 entries of the row's table, two to a lane, from entry 32 `win`
        PagedAt ahead = at;
        int2 who = row_at(at.row);
        int win, ent0, ent1;
        auto entries = [&](int w) {
            const int e = 32 * w + lane;
            return e < a.width ? __ldcg(a.table + (int64_t)who.x * a.width + e) : -1;
        };
        auto open = [&](int w) {
            win = w;
            ent0 = entries(w);
            ent1 = entries(w + 1);
        };
        open(page_of(at.st * KS) >> 5);
        // the lane's slot of the cache in the stage `ahead` (-1: hidden) and its kv head; then on to the next stage
        int g_ahead = 0;
        auto place = [&]() {
            const int slot = ahead.st * KS + (KS == 32 ? lane : lane & 15), pg = page_of(slot), off = slot - pg * a.page;
            const int w = __shfl_sync(0xffffffffu, pg, 0) >> 5;
            if (w != win) {  // (a stage has at most 32 pages)
                if (w == win + 1) {
                    win = w;
                    ent0 = ent1;
                    ent1 = entries(w + 1);
                } else {
                    open(w);
                }
            }
            const int e0 = __shfl_sync(0xffffffffu, ent0, pg & 31), e1 = __shfl_sync(0xffffffffu, ent1, pg & 31);
            const int entry = (pg >> 5) == win ? e0 : e1;
            const int phys = slot <= who.y && entry >= 0 && entry < a.n_pages ? entry * a.page + off : -1;
            g_ahead = ahead.gi / HT;
            if (++ahead.st == ahead.nst) {
                ahead.st = 0;
                if (++ahead.gi == GI) {
                    ahead.gi = 0;
                    const int r = next_row(ahead.row);
                    if (r < a.n && fetch > 1) {
                        ahead.row = r;
                        ahead.nst = first[r + 1] - first[r];
                        who = row_at(r);
                        open(0);
                    }
                }
            }
            return phys;
        };
        auto rows_in = [&](const void* base, int phys, bool whole, uint32_t dst, bool isv) {
            constexpr int CPR = C::RB / 16, RPI = CPR <= 32 ? 32 / CPR : 1, N = 16 / RPI;  // rows of an instruction, instructions of 16
            static_assert(CPR <= 32 && N * RPI == 16, "");
            const uint8_t* src = (const uint8_t*)base + (int64_t)g_ahead * a.c.ctx * C::RB + lane % CPR * 16;
            const int r0 = lane / CPR;
            dst += (isv ? C::vbyte(r0, lane % CPR * 16) : C::kbyte(r0, lane % CPR * 16));
            auto to = [&](int x, int i) {  // (swizzles are linear in the bits of the row)
                const int sw = isv ? C::swv(i * RPI) : C::swk(i * RPI);
                return (dst ^ (sw << 4)) + (16 * x + i * RPI) * C::RB;
            };
            if (whole) {  // 16 slots are neighbours in memory
#pragma unroll
                for (int x = 0; x < SUB; x++) {
                    const uint8_t* p = src + ((int64_t)__shfl_sync(0xffffffffu, phys, 16 * x) + (isv ? r0 : C::kslot(r0))) * C::RB;
#pragma unroll
                    for (int i = 0; i < N; i++) copy16(to(x, i), p + (isv ? i * RPI : C::kslot(i * RPI)) * C::RB, 16);
                }
            } else {
#pragma unroll
                for (int x = 0; x < SUB; x++)
#pragma unroll
                    for (int i = 0; i < N; i++) {
                        const int p = __shfl_sync(0xffffffffu, phys, 16 * x + (isv ? r0 + i * RPI : C::kslot(r0) + C::kslot(i * RPI)));
                        copy16(to(x, i), src + (int64_t)max(p, 0) * C::RB, p >= 0 ? 16 : 0);
                    }
            }
        };
        // the 16 bytes around the scales of the lane's slot (up to the last scale of the cache)
        auto scales_in = [&](const __half* base, int phys, uint32_t dst) {
            if constexpr (C::QUANT) {
                const int64_t row = (int64_t)g_ahead * a.c.ctx + max(phys, 0), end = (int64_t)KVH * a.c.ctx * C::SB;
                const int64_t from = row * C::SB & ~(int64_t)15;
                copy16(dst + 16 * lane, (const uint8_t*)base + from, phys < 0 ? 0 : (int)min(end - from, (int64_t)16));
            }
        };
        bool whole = false;  // of the stage: all slots are seen, and pages hold 16 at a time
        auto fetch_k = [&](int phys, int slot) {
            const uint32_t dst = ring + slot * C::STAGE;
            const unsigned see = __ballot_sync(0xffffffffu, phys >= 0);
            whole = see == 0xffffffffu && a.page % 16 == 0;
            rows_in(a.c.k, phys, whole, dst, false);
            scales_in(a.c.ks, phys, dst + C::OKS);
            unsigned b0 = 0, b1 = 0;
            if constexpr (C::QUANT) {
                const unsigned row = (unsigned)g_ahead * (unsigned)a.c.ctx + (unsigned)phys;
                b0 = __ballot_sync(0xffffffffu, row & 1);
                if (NB == 2) b1 = __ballot_sync(0xffffffffu, row & 2);
            }
            if (lane == 0) sm_head[warp][slot] = make_uint4(see, b0, b1, 0u);
        };
        auto fetch_v = [&](int phys, int slot) {
            const uint32_t dst = ring + slot * C::STAGE;
            rows_in(a.c.v, phys, whole, dst, true);
            scales_in(a.c.vs, phys, dst + C::OVS);
        };
        // codes: where this lane's rows of the matrices of K and V begin
        constexpr int CPR = C::RB / 16;
        const int kaddr = CPR >= 4 ? C::kbyte(lane & 7, (lane >> 3) * 16) : C::kbyte((lane & 7) + 8 * (lane >> 4), (lane >> 3 & 1) * 16);
        const int vaddr = C::vbyte(lane & 15, (lane >> 4) * 16) - C::OV;

        // The counters of the items that this CTA may hold a part of: that of its first stage and the one that begins in it.
        // A counter holds the call's mark and the number of pieces left; what has another mark is nothing (below).
        unsigned long long* const mine = counters + (lane ? (int)blockIdx.x : cta_of(begin_unit + u - at.st));
        unsigned long long found = 0;
        if (warp == 0 && lane < 2) found = __ldcg(mine);

        uint32_t qf[NT][C::STEPS][2];  // q's operands
        float rowf[NT];
        float o[NT][C::MT][4], m_ref[NT], l[NT];
        bool seen = false, begun = true;  // begun: the piece begins with its item
        bool fresh = true;
        int slot = 0;
        // The first NST rounds only fetch; after them a stage is computed before its place takes the stage NST ahead.
        for (int round = -NST;; round++) {
            const bool work = round >= 0;
            const int g = at.gi / HT, ht = at.gi - g * HT;
            const uint32_t st = ring + slot * C::STAGE;
            unsigned see = 0;  // the stage's slots that are seen
            float s[NT][SUB][2];  // scores: this lane's slots j and j + 8 of each 16, head c of tile t
            int so[SUB][2];  // where the scales of this lane's slots lie
            auto scale = [&](uint32_t base, int x, int h, uint32_t (&w)[2]) {  // the words of blocks 0, 1 and 2, 3
                if (NB == 4) {
                    shared64(base + so[x][h], w);
                } else {
                    w[0] = shared32(base + so[x][h]);
                    w[1] = 0;
                }
            };
            if (work) {
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
                            const int d = TYPE == AF_F32 || TYPE == AF_KV_Q8_0 ? 16 * i + 4 * c : 32 * (i >> 1) + 8 * c + 4 * (i & 1);
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
                                    qf[t][2 * i + (e >> 1)][e & 1] = part ? lo : hi;
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
                }
                copy_wait<2 * NST - 1>();
                __syncwarp();  // every lane's copies of this stage's K have landed
                asm volatile("" ::: "memory");
                const uint4 hd = sm_head[warp][slot];
                see = hd.x;
                if constexpr (C::QUANT) {
#pragma unroll
                    for (int x = 0; x < SUB; x++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int i = 16 * x + C::slot(h, j);
                            so[x][h] = st + 16 * i + (NB == 4 ? (hd.y >> i & 1) * 8 : (hd.y >> i & 1) * 4 + (hd.z >> i & 1) * 8);
                        }
                }
                // ---- scores
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int x = 0; x < SUB; x++) s[t][x][0] = s[t][x][1] = 0.f;
#pragma unroll
                for (int x = 0; x < SUB; x++) {
                    uint32_t dk[2][2];
                    uint32_t kc[2][2 * NB];  // codes: a word of each 16 bytes of the rows j of both halves
                    if constexpr (C::QUANT) {
                        scale(C::OKS, x, 0, dk[0]);
                        scale(C::OKS, x, 1, dk[1]);
                        constexpr int CPR = C::RB / 16;
                        if constexpr (CPR >= 4) {
#pragma unroll
                            for (int h = 0; h < 2; h++)
#pragma unroll
                                for (int g4 = 0; g4 < CPR; g4 += 4)
                                    rows4(st + (kaddr ^ (g4 << 4)) + (16 * x + 8 * h) * C::RB, &kc[h][g4]);
                        } else {  // (both halves' two chunks)
                            uint32_t y[4];
                            rows4(st + kaddr + 16 * x * C::RB, y);
                            kc[0][0] = y[0], kc[0][1] = y[1], kc[1][0] = y[2], kc[1][1] = y[3];
                        }
                    }
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        if constexpr (TYPE == AF_F32) {
                            float p[NT][4] = {};
                            uint32_t hi[2][8], lo[2][8];
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                shared128(st + C::kbyte(8 * h + j, (8 * b + c) * 16), hi[h]);
                                shared128(st + C::kbyte(8 * h + j, (8 * b + 4 + c) * 16), hi[h] + 4);
#pragma unroll
                                for (int i = 0; i < 8; i++) cut_tf32(__uint_as_float(hi[h][i]), hi[h][i], lo[h][i]);
                            }
#pragma unroll
                            for (int e = 0; e < 8; e++) {  // the small lo products first
                                const int i = 2 * (e & 3), step = 4 * b + (e & 3);
                                const uint32_t *k0 = e < 4 ? lo[0] : hi[0], *k1 = e < 4 ? lo[1] : hi[1];
#pragma unroll
                                for (int t = 0; t < NT; t++)
                                    dot8(p[t], make_uint4(k0[i], k1[i], k0[i + 1], k1[i + 1]), qf[t][step][0], qf[t][step][1]);
                            }
#pragma unroll
                            for (int t = 0; t < NT; t++) s[t][x][0] += p[t][0] + p[t][1], s[t][x][1] += p[t][2] + p[t][3];
                        } else {
                            uint32_t w[2][4];
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                if constexpr (TYPE == AF_F16) {
                                    shared128(st + C::kbyte(16 * x + 8 * h + j, (4 * b + c) * 16), w[h]);
                                } else if constexpr (TYPE == AF_KV_Q8_0) {
#pragma unroll
                                    for (int i = 0; i < 2; i++) codes2(kc[h][2 * b + i], w[h][2 * i], w[h][2 * i + 1]);
                                } else {
                                    codes4(kc[h][b], w[h]);
                                }
                            }
#pragma unroll
                            for (int t = 0; t < NT; t++) {
                                float p[4];
                                dot16z(p, make_uint4(w[0][0], w[1][0], w[0][1], w[1][1]), qf[t][2 * b][0], qf[t][2 * b][1]);
                                dot16(p, make_uint4(w[0][2], w[1][2], w[0][3], w[1][3]), qf[t][2 * b + 1][0], qf[t][2 * b + 1][1]);
                                const float s0 = p[0] + p[1], s1 = p[2] + p[3];
                                if constexpr (C::QUANT) {
                                    const __half2 d0 = u_h2(dk[0][b / 2]), d1 = u_h2(dk[1][b / 2]);
                                    s[t][x][0] = fmaf(__half2float(b & 1 ? __high2half(d0) : __low2half(d0)), s0, s[t][x][0]);
                                    s[t][x][1] = fmaf(__half2float(b & 1 ? __high2half(d1) : __low2half(d1)), s1, s[t][x][1]);
                                } else {
                                    s[t][x][0] += s0;
                                    s[t][x][1] += s1;
                                }
                            }
                        }
                    }
                }
            }
            // ---- K's place in the ring takes the stage NST ahead
            int phys = -1;
            __syncwarp();
            if (fetch > 0) {
                phys = place();
                fetch_k(phys, slot);
            }
            copy_commit();
            if (work) {
                copy_wait<2 * NST - 1>();
                __syncwarp();  // V has landed
                asm volatile("" ::: "memory");
                uint32_t vs[SUB][2][2];
                if constexpr (C::QUANT) {
#pragma unroll
                    for (int x = 0; x < SUB; x++)
#pragma unroll
                        for (int h = 0; h < 2; h++) scale(C::OVS, x, h, vs[x][h]);
                }
                // ---- softmax; hidden slots have no score (and zeros as values)
                seen |= see != 0;
                if (see != 0xffffffffu) {
#pragma unroll
                    for (int x = 0; x < SUB; x++)
#pragma unroll
                        for (int h = 0; h < 2; h++)
                            if (!(see >> (16 * x + C::slot(h, j)) & 1)) {
#pragma unroll
                                for (int t = 0; t < NT; t++) s[t][x][h] = -CUDART_INF_F;
                            }
                }
                float big[SUB][2];  // log2 of the slots' largest value scales
                if constexpr (C::QUANT) {
#pragma unroll
                    for (int x = 0; x < SUB; x++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            __half2 m = __habs2(u_h2(vs[x][h][0]));
                            if (NB == 4) m = __hmax2(m, __habs2(u_h2(vs[x][h][1])));
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
                    for (int y = 0; y < D / 32; y++) {  // dims 32 y + 4 j .. + 3: two row tiles
                        uint32_t lo[4][4], hi[4][4];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            shared128(st + C::vbyte(c + 4 * k, (8 * y + j) * 16), hi[k]);
#pragma unroll
                            for (int e = 0; e < 4; e++) cut_tf32(__uint_as_float(hi[k][e]), hi[k][e], lo[k][e]);
                        }
#pragma unroll
                        for (int t = 0; t < NT; t++)
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                float sum[4];
                                dot8z(sum, make_uint4(lo[0][e], lo[0][e + 1], lo[1][e], lo[1][e + 1]), pb[t][0][0], pb[t][0][1]);
                                dot8(sum, make_uint4(lo[2][e], lo[2][e + 1], lo[3][e], lo[3][e + 1]), pb[t][1][0], pb[t][1][1]);
                                dot8(sum, make_uint4(hi[0][e], hi[0][e + 1], hi[1][e], hi[1][e + 1]), pb[t][0][0], pb[t][0][1]);
                                dot8(sum, make_uint4(hi[2][e], hi[2][e + 1], hi[3][e], hi[3][e + 1]), pb[t][1][0], pb[t][1][1]);
                                add4(o[t][2 * y + e / 2], sum);
                            }
                    }
                } else if constexpr (TYPE == AF_F16) {
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int t = 0; t < NT; t++)
#pragma unroll
                        for (int h = 0; h < 2; h++) pb[t][h] = transpose8(hi_lo(s[t][0][h]));
#pragma unroll
                    for (int y = 0; y < D / 64; y++) {  // dims 64 y + 8 j .. + 7: four row tiles
                        uint32_t w[4][4];
#pragma unroll
                        for (int k = 0; k < 4; k++) shared128(st + C::vbyte(2 * c + (k & 1) + 8 * (k >> 1), (8 * y + j) * 16), w[k]);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const uint4 v = make_uint4(__byte_perm(w[0][i], w[1][i], 0x5410), __byte_perm(w[0][i], w[1][i], 0x7632),
                                                       __byte_perm(w[2][i], w[3][i], 0x5410), __byte_perm(w[2][i], w[3][i], 0x7632));
#pragma unroll
                            for (int t = 0; t < NT; t++) {
                                float sum[4];
                                dot16z(sum, v, pb[t][0], pb[t][1]);
                                add4(o[t][4 * y + i], sum);
                            }
                        }
                    }
                } else {
                    uint32_t vc[SUB][4];
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        uint32_t pb[NT][SUB][2];
#pragma unroll
                        for (int x = 0; x < SUB; x++) {
                            float d[2];
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const __half2 w = u_h2(vs[x][h][b / 2]);
                                d[h] = __half2float(b & 1 ? __high2half(w) : __low2half(w));
                            }
#pragma unroll
                            for (int t = 0; t < NT; t++) {  // p d in two parts, of two slots at a time
                                const float2 y = mul2(make_float2(s[t][x][0], s[t][x][1]), make_float2(d[0], d[1]));
                                const float2 hi = make_float2(__uint_as_float(__float_as_uint(y.x) & 0xFFFFE000u), __uint_as_float(__float_as_uint(y.y) & 0xFFFFE000u));
                                const float2 lo = fma2(hi, both(-1.f), y);
                                pb[t][x][0] = transpose8(h2_u(__floats2half2_rn(hi.x, lo.x)));
                                pb[t][x][1] = transpose8(h2_u(__floats2half2_rn(hi.y, lo.y)));
                            }
                        }
                        float sum[NT][2][4];
#pragma unroll
                        for (int x = 0; x < SUB; x++) {
                            uint32_t v[2][4];  // pair of slots, row of the two row tiles
                            if constexpr (TYPE == AF_KV_Q8_0) {
                                uint32_t y[4];  // dims j, j + 8, j + 16, j + 24 of four slots
                                columns4(st + C::OV + (vaddr ^ (b << 5)) + 16 * x * C::RB, y);
#pragma unroll
                                for (int i = 0; i < 4; i++) codes2(y[i], v[0][i], v[1][i]);
                            } else {
                                if (b % 2 == 0) columns4(st + C::OV + (vaddr ^ (b << 4)) + 16 * x * C::RB, vc[x]);  // two blocks' bytes
#pragma unroll
                                for (int i = 0; i < 2; i++) {  // bytes j and j + 8 of the block: dims 2j, 2j + 1 and 16 more
                                    const uint32_t y = vc[x][2 * (b & 1) + i], lo = y & 0x0F0F0F0Fu, hi = y & 0xF0F0F0F0u;
                                    const __half2 f = __float2half2_rn(0.0625f), m72 = __float2half2_rn(-72.f);  // (1024 + 16 n) / 16 - 72
                                    v[0][2 * i] = hsub2u(__byte_perm(lo, 0x64646464u, 0x4140), 0x64086408u);
                                    v[1][2 * i] = hsub2u(__byte_perm(lo, 0x64646464u, 0x4342), 0x64086408u);
                                    v[0][2 * i + 1] = h2_u(__hfma2(u_h2(__byte_perm(hi, 0x64646464u, 0x4140)), f, m72));
                                    v[1][2 * i + 1] = h2_u(__hfma2(u_h2(__byte_perm(hi, 0x64646464u, 0x4342)), f, m72));
                                }
                            }
#pragma unroll
                            for (int t = 0; t < NT; t++)
#pragma unroll
                                for (int i = 0; i < 2; i++) {
                                    const uint4 w = make_uint4(v[0][2 * i], v[0][2 * i + 1], v[1][2 * i], v[1][2 * i + 1]);
                                    if (x == 0)
                                        dot16z(sum[t][i], w, pb[t][x][0], pb[t][x][1]);
                                    else
                                        dot16(sum[t][i], w, pb[t][x][0], pb[t][x][1]);
                                }
                        }
#pragma unroll
                        for (int t = 0; t < NT; t++)
#pragma unroll
                            for (int i = 0; i < 2; i++) add4(o[t][2 * b + i], sum[t][i]);
                    }
                }
            }
            // ---- V's place in the ring takes the stage NST ahead
            __syncwarp();
            if (fetch > 0) {
                fetch--;
                fetch_v(phys, slot);
            }
            copy_commit();
            slot = slot + 1 == NST ? 0 : slot + 1;
            if (!work) {
                // (one try: where it fails, another CTA of the item has set the mark)
                if (round == -1 && warp == 0 && lane < 2 && found >> 16 != a.mark) atomicCAS(mine, found, a.mark << 16);
                continue;
            }

            // ---- the end of the item, or of this warp's range
            const bool ends = at.st + 1 == at.nst;
            if (ends || left == 1) {
                fresh = true;
                const bool done = begun && ends;
                const int which = begun ? 1 : 0;
                float* piece = left == 1 ? my_piece : far + warp * C::PIECE;  // (all copies are done)
                if (!done && lane == 0) sm_piece[warp][which] = make_int4(at.row, at.gi, left == 1 ? 1 : 2, ends);
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
                        if constexpr (C::QUANT) {
#pragma unroll
                            for (int i = 0; i < C::MT; i++) {
                                const float y = (o[t][i][0] + o[t][i][1]) * inv, z = (o[t][i][2] + o[t][i][3]) * inv;
                                if (TYPE == AF_KV_Q8_0) {  // rows j and j + 8 are dims 16 i + j and 8 on
                                    dst[16 * i + j] = y;
                                    dst[16 * i + 8 + j] = z;
                                } else {
                                    *reinterpret_cast<float2*>(dst + 16 * i + 2 * j) = make_float2(y, z);
                                }
                            }
                        } else {
                            // row tile i: dims (j) and (j + 8) of its output are neighbours, i and i + 1 make four
#pragma unroll
                            for (int i = 0; i < C::MT; i += 2) {
                                const int d = TYPE == AF_F16 ? 64 * (i >> 2) + 8 * j + 2 * (i & 3) : 32 * (i >> 1) + 4 * j;
                                *reinterpret_cast<float4*>(dst + d) =
                                    make_float4((o[t][i][0] + o[t][i][1]) * inv, (o[t][i][2] + o[t][i][3]) * inv,
                                                (o[t][i + 1][0] + o[t][i + 1][1]) * inv, (o[t][i + 1][2] + o[t][i + 1][3]) * inv);
                            }
                        }
                    }
                }
            }
            if (ends) {
                at.st = 0;
                if (++at.gi == GI) {
                    at.gi = 0;
                    if (left > 1) {
                        at.row = next_row(at.row);
                        at.nst = first[at.row + 1] - first[at.row];
                    }
                }
            } else {
                at.st++;
            }
            if (--left == 0) break;
        }
    }

    // ---- join: chains of pieces in the order of the warps; a warp takes every NW-th head of all chains
    __syncthreads();
    float* const pieces = a.ws + paged_pieces(gridDim.x);
    int4 p0 = make_int4(0, 0, 0, 0), p1 = p0;  // lane x: the pieces of warp x
    if (lane < NW) p0 = sm_piece[lane][0], p1 = sm_piece[lane][1];
    const unsigned used0 = __ballot_sync(0xffffffffu, p0.z != 0), ends0 = __ballot_sync(0xffffffffu, p0.z && p0.w);
    unsigned heads1 = __ballot_sync(0xffffffffu, p1.z != 0);  // warps in which a chain begins
    const float* const near_by = reinterpret_cast<const float*>(smem + min(lane, NW - 1) * NST * C::STAGE);
    const float* const far_off = far + min(lane, NW - 1) * C::PIECE;
    int job = warp;                                             // heads before this warp's next one
    int4 own0 = make_int4(0, 0, 0, 0), own1 = own0;  // items of which the CTA leaves pieces 0 and 1 (.z: it does)
    // A piece 0 goes on with an earlier warp's item; the CTA's first one goes on with another CTA's.
    const unsigned cta0 = used0 & -used0 & (heads1 ? (heads1 & -heads1) * 2 - 1 : ~0u);
#pragma unroll 1
    for (int slot = cta0 ? 0 : 1; slot == 0 || heads1; slot = 1) {
        const int w = __ffs(slot ? heads1 : cta0) - 1;
        if (slot) heads1 &= heads1 - 1;
        const int4 pw = slot ? p1 : p0;
        const int4 p = make_int4(__shfl_sync(0xffffffffu, pw.x, w), __shfl_sync(0xffffffffu, pw.y, w), __shfl_sync(0xffffffffu, pw.z, w),
                                 __shfl_sync(0xffffffffu, pw.w, w));
        const unsigned above = used0 & ~((2u << w) - 1), stop = ends0 & above;
        const bool here = slot == 0 && p.w;  // it ends where it begins
        const unsigned more = here ? 0 : stop ? above & ((stop & -stop) * 2 - 1) : above;  // the other warps of the chain
        const bool out = slot == 1 && more && stop;
        if (!out) (slot ? own1 : own0) = p;
        const int g = p.y / HT, ht = p.y - g * HT;
        const float* const mine = (lane == w ? pw.z : p0.z) == 1 ? near_by : far_off;
        const unsigned chain = more | 1u << w;
#pragma unroll 1
        for (; job < C::HEADS; job += NW) {
            const int hh = job, head = ht * C::HEADS + hh;
            if (head >= G) continue;
            float2 ml = make_float2(-CUDART_INF_F, 0.f);
            if (chain >> lane & 1) ml = reinterpret_cast<const float2*>(mine + C::HEADS * D)[hh];
            float m = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            // A piece that saw nothing adds nothing; one that saw only scores of -infinity has weights of zero, which a value that is
            // not finite turns into NaN.
            const bool none = __float_as_uint(ml.y) == 0;
            const float f = ml.x == -CUDART_INF_F ? 0.f : ex2t(ml.x - m);
            float den = f * ml.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
            const bool saw = __any_sync(0xffffffffu, __float_as_uint(ml.y) != 0);
            const unsigned adds = __ballot_sync(0xffffffffu, !none);
            float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
            float4 v[4];
            float fx[4];
            for (unsigned rest = adds; rest;) {  // four pieces' loads at a time
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int x = rest ? __ffs(rest) - 1 : 0;
                    const float* src = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, (unsigned long long)mine, x));
                    const float fs = __shfl_sync(0xffffffffu, f, x);
                    const bool in = rest != 0;
                    fx[i] = in ? fs : 0.f;
                    v[i] = in && 4 * lane < D ? *reinterpret_cast<const float4*>(src + hh * D + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
                    rest &= rest - 1;
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
                    num.x += fx[i] * v[i].x, num.y += fx[i] * v[i].y, num.z += fx[i] * v[i].z, num.w += fx[i] * v[i].w;
            }
            if (out) {
                const float inv = den != 0.f ? 1.f / den : saw ? CUDART_NAN_F : 0.f;
                if (4 * lane < D)
                    *reinterpret_cast<float4*>(a.out + (int64_t)p.x * a.ldo + (int64_t)(g * G + head) * D + 4 * lane) =
                        make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
            } else {
                float* dst = pieces + (size_t)(blockIdx.x * 2 + slot) * paged_piece_floats(D);
                if (4 * lane < D) *reinterpret_cast<float4*>(dst + hh * D + 4 * lane) = num;
                if (den == 0.f && saw) den = -0.f;
                if (lane == 0) reinterpret_cast<float2*>(dst + kPagedHeads * D)[hh] = make_float2(m, den);
            }
        }
        job -= C::HEADS;
    }
    if (!own0.z && !own1.z) {
        __threadfence();
        return;
    }
    // ---- items of several CTAs: the last CTA to leave its piece joins them, in order
    __shared__ int2 sm_chain[2];  // first and last CTA of an item that this one joins; first < 0: it does not
    const int4 mine_of = tid ? own1 : own0;
    int2 chain = make_int2(0, 0);
    if (tid < 2 && mine_of.z) {
        const int64_t nst = first[mine_of.x + 1] - first[mine_of.x], from = begin_unit + (int64_t)first[mine_of.x] * GI + mine_of.y * nst;
        chain = make_int2(cta_of(from), cta_of(from + nst - 1));
    }
    __syncthreads();
    if (tid < 2) {
        unsigned long long left = ~0ull;
        if (mine_of.z)  // (the barrier has put the CTA's pieces before this thread, the release puts them before the count)
            asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], 1;" : "=l"(left) : "l"(counters + chain.x) : "memory");
        if ((int)(left & 0xFFFF) == chain.y - chain.x)
            counters[chain.x] = 0;
        else
            chain = make_int2(-1, -1);
        sm_chain[tid] = chain;
    }
    __syncthreads();
    // a warp takes every NW-th head of one or two items; sums over 32 pieces at a time
#pragma unroll 1
    for (int x = warp; x < 2 * C::HEADS; x += NW) {
        const int which = x / C::HEADS, hh = x % C::HEADS;
        const int2 chain = sm_chain[which];
        const int4 p = which ? own1 : own0;
        const int n = chain.y - chain.x + 1, g = p.y / HT, head = (p.y - g * HT) * C::HEADS + hh, d = 4 * lane < D ? 4 * lane : 0;
        if (chain.x < 0 || head >= G) continue;
        auto piece = [&](int i) { return pieces + (size_t)(2 * (chain.x + i) + (i ? 0 : 1)) * paged_piece_floats(D); };
        float m = -CUDART_INF_F, den = 0.f;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        bool saw = false;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += 32) {
            float2 ml = make_float2(-CUDART_INF_F, 0.f);
            if (i0 + lane < n) ml = __ldcg(reinterpret_cast<const float2*>(piece(i0 + lane) + kPagedHeads * D) + hh);
            float4 v[8];
            auto load = [&](int k0) {
#pragma unroll
                for (int k = 0; k < 8; k++)
                    if (i0 + k0 + k < n) v[k] = __ldcg(reinterpret_cast<const float4*>(piece(i0 + k0 + k) + hh * D + d));
            };
            load(0);
            float top = fmaxf(m, ml.x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (top > m) {
                const float f = ex2t(m - top);
                m = top;
                den *= f, num.x *= f, num.y *= f, num.z *= f, num.w *= f;
            }
            const bool none = __float_as_uint(ml.y) == 0;  // (as above)
            const float f = ml.x == -CUDART_INF_F ? 0.f : ex2t(ml.x - m);
            float sum = f * ml.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            den += sum;
            saw |= __any_sync(0xffffffffu, __float_as_uint(ml.y) != 0);
            const unsigned adds = __ballot_sync(0xffffffffu, !none);
#pragma unroll 1
            for (int k0 = 0; k0 < 32 && i0 + k0 < n; k0 += 8) {
                if (k0) load(k0);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float w = __shfl_sync(0xffffffffu, f, k0 + k);
                    if (adds >> (k0 + k) & 1) num.x += w * v[k].x, num.y += w * v[k].y, num.z += w * v[k].z, num.w += w * v[k].w;
                }
            }
        }
        const float inv = den != 0.f ? 1.f / den : saw ? CUDART_NAN_F : 0.f;
        if (4 * lane < D)
            *reinterpret_cast<float4*>(a.out + (int64_t)p.x * a.ldo + (int64_t)(g * G + head) * D + 4 * lane) =
                make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
    }
    __threadfence();  // (and no early launch of the next kernel: the rows may be a cache, see launch_chained)
}

// One translation unit per cache type.
template <int TYPE>
cudaError_t launch_attn_paged_type(const PagedArgs& a, int ctas, cudaStream_t s);

template <int TYPE, int D, int NT>
cudaError_t paged_go(const PagedArgs& a, int ctas, cudaStream_t s) {
    using C = PagedCfg<TYPE, D, NT>;
    static_assert(C::NW * C::PIECE <= 8 * paged_piece_floats(D), "workspace");
    auto k = attn_paged_kernel<TYPE, D, NT>;
    static SmemOptIn opt;
    cudaError_t e = opt((const void*)k, C::FIXED + C::ROWS);
    if (e) return e;
    return launch_chained(k, dim3(ctas), C::NW * 32, C::FIXED + (a.n + 1) * 4 + (a.n <= kPagedKept ? a.n * 8 : 0), s, a);
}

#define AF_PAGED_INSTANTIATE(TYPE)                                                                    \
    template <>                                                                                       \
    cudaError_t launch_attn_paged_type<TYPE>(const PagedArgs& a, int ctas, cudaStream_t s) {          \
        const int G = a.H / a.c.KVH;                                                                  \
        if (a.c.D == 64) return G > 4 ? paged_go<TYPE, 64, 2>(a, ctas, s) : paged_go<TYPE, 64, 1>(a, ctas, s); \
        return G > 4 ? paged_go<TYPE, 128, 2>(a, ctas, s) : paged_go<TYPE, 128, 1>(a, ctas, s);       \
    }

}  // namespace af

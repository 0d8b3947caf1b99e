// Tree attention (attn_tree.cu has the definition) on the 5th-generation tensor cores, for calls with more rows than
// one mma.sync tile pair.
//
// CTA (split, kv head g, row tile): 128 rows (row = node G + head of the group) are the 128 TMEM lanes.  With
// everything that belongs to a row in tensor memory (q, scores, p and the output: 512 columns), shared memory holds
// only K and V operands, and an MMA reads nothing else from it:
//   columns [0, D)          output accumulator of up to kFlush tiles, fp32
//   columns [D, 2 D)        the output of the tiles before them
//   columns [2 D, 3 D)      q, scaled by log2 e / sqrt(D) and a power of two per row, as fp16 hi and lo parts
//   columns [3 D + 64 b..)  scores of a tile (64 fp32 columns, b < 2 or, with D = 64, 4), overwritten, 32 slots by 32, by
//                           p's fp16 hi and lo parts (16 columns each)
// The tensor cores' fp32 sums are cut, not rounded: every product added to a sum takes up to 2^-23 of it, always towards
// zero.  So the small lo products come first, before the sum has its size, and the output is added to the older tiles'
// by the softmax warps, rounded, every kFlush tiles (64 nodes over 30720 fp32 slots are off by 1.2e-5 of the result's
// norm with one sum of 53 tiles, in 108.7 us; sums of 4, 2 and 1 tiles: 1.2e-6 in 109.9, 8.1e-7 in 111.3, 6.5e-7 in 113.8).
// Both products take their A operand (q, p) from tensor memory and B from shared memory: K rows [slot][dim] are
// K-major, V rows [slot][dim] MN-major, so neither is transposed and both have the cache's own order:
//   fp16 cache    TMA copies 64 slots x 64 dims boxes into the SWIZZLE_128B layout; two products (hi, lo of q or p)
//   fp32, Q8_0, Q4_0  bulk copies bring the raw rows into a staging ring, four warps for K and four for V write them
//                 as fp16 hi and lo parts in the same layout; three products (the dropped lo lo is 2^-22 relative).
//                 Sixteen slots are scaled by a power of two that brings their largest value (or scale) near 1, so
//                 fp16's range never binds; where the slots' own largest values are more than 2^kSpread apart, each slot
//                 by its own (one large key, hidden or not, would leave its neighbours few bits).  K's power goes into
//                 the scores; V's into p, relative to a reference exponent of the row's output, which is rescaled when
//                 p times V, over the slots that the row sees, outgrows it.
//                 (Rows read through registers instead, three tiles ahead: 1.8 times as long at 64 nodes over 30720
//                 fp32 slots; the warp's loads of several tiles share its few scoreboards.)
// Warps 0-7 are the softmax: a thread owns a row and 32 of a tile's slots (its scores in registers: maximum, p, sum), the
// two of a row exchange their maxima tile by tile.  (One thread for all 64 slots was the longest chain of the pipeline:
// some 500 instructions a tile and a warp beside eight converting warps: 25 nodes over 30011 Q8_0 slots took 6% longer.)
// One warp issues the MMAs, scores two (D = 64: three) tiles ahead of the outputs.
// The reference maximum moves lazily, as in attn_tree.cu, with the same factor 2^8 in p.
// Tiles that hold nodes (the last ones): a hidden slot's score is -inf by a select; non-finite keys and values and the
// slots behind the last node become zero operands, and a row that sees a slot so treated becomes NaN.
// Every wait is bounded: a CTA that gives up lets what it issued finish, frees its TMEM and marks its rows NaN.
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "draft.cuh"
#include "tcgen05.cuh"

namespace af {

namespace {

constexpr int BK = 64;         // slots per tile
constexpr int kFlush = 2;      // tiles of one output sum
constexpr int kTmem = 512;
constexpr int kQueueBar = 1;   // named barrier: q has been read
constexpr int kRows = 128;
constexpr float kLazy2 = 4.f, kBias2 = 8.f;  // as attn_tree.cu's
constexpr int kConvWarps = 4;  // for K, and as many for V: 16 slots of a tile each
constexpr int kNoExp = -128, kMaxExp = 126;  // exponents of slots: of zeros, and the largest (an infinity's too)
constexpr float kNoRef = -1000.f;  // the output's reference exponent before it has one
constexpr int kSpread = 3;     // 16 slots whose exponents differ by more than this have their own
constexpr int kSoftWarps = 8;  // two per 32 rows

template <int TYPE, int D>
struct TcCfgT {
    static constexpr bool SPLIT = TYPE != AF_F16;
    static constexpr int ACC = D, QCOL = 2 * D, SCOL = 3 * D;    // tensor memory columns
    static constexpr int SB = D == 128 ? 2 : 4;               // score buffers (what is left of tensor memory)
    static constexpr int AHEAD = D == 128 ? 2 : 3;            // tiles whose scores are issued ahead of the outputs
    static_assert(SCOL + SB * BK <= kTmem, "tensor memory");
    static constexpr int PART = BK * D * 2;                  // one fp16 operand of a tile
    static constexpr int SLOT = PART * (SPLIT ? 2 : 1);      // hi (and lo)
    static constexpr int NS = SPLIT ? (D == 128 ? 2 : 4) : 6;  // operand slots of K, and of V
    // staging of raw rows: RR rows a slot, NR slots for K and for V
    static constexpr int RB = TYPE == AF_F32 ? 4 * D : TYPE == AF_KV_Q8_0 ? D : D / 2;
    static constexpr int SCB = TYPE == AF_F32 ? 0 : D / 16;  // scale bytes of a row
    static constexpr int RR = TYPE == AF_F32 ? BK / 2 : BK, RU = RR / 16;  // (the rows of RU warps)
    static constexpr int RAW = RR * (RB + SCB);
    static constexpr int NR = !SPLIT ? 0 : TYPE == AF_F32 ? (D == 128 ? 3 : 5) : 5;
    // tiles whose K exponents are kept: while the softmax is at tile t, the scores of t + AHEAD - 1 may be done and the
    // converters at the tile NS after that
    static constexpr int EK = !SPLIT ? 1 : D == 128 ? 4 : 8;
    static_assert(!SPLIT || AHEAD + NS <= EK, "exponents of K are read before they are overwritten");
    static constexpr int OFF_V = NS * SLOT, OFF_RAW = 2 * NS * SLOT;
    static constexpr int QS = kRows * D * 4 / SLOT;          // the last V slots, through which q and the output pass
    static_assert(QS <= NS, "q fits the V slots");
    static constexpr int MMA_WARP = kSoftWarps + (SPLIT ? 2 * kConvWarps : 0), COPY_WARP = MMA_WARP + 1;  // + 1: V's copies
    static constexpr int WARPS = COPY_WARP + 2;
    // at least more than half of an SM's shared memory: a CTA takes all of its tensor memory
    static constexpr int USED = OFF_RAW + 2 * NR * RAW;
    static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
};

// Of pairs, [0] is K's and [1] V's.
template <typename C>
struct alignas(1024) TcState {  // (the operand slots behind it need 1024 bytes)
    static constexpr int NR = C::NR ? C::NR : 1, NE = C::SPLIT ? C::NS : 1;
    // by tile and 16 slots, K's 2^exponent (infinity: the slots have exponents of their own); by operand slot, V's exponent
    // (infinity likewise, NaN: zeros)
    float kf[C::EK][4], vf[NE][4];
    int8_t ek[C::EK][BK], ev[NE][BK];  // the slots' exponents (kNoExp: zeros)
    uint64_t full[2][C::NS], empty[2][C::NS];  // operand slots
    uint64_t raw_full[2][NR], raw_empty[2][NR];  // staging slots
    uint64_t s_full[C::SB], p_full[C::SB], pv_done[C::SB];
    uint64_t q_ready, done;
    uint64_t v_clean;                          // fp16: a tile of nodes has its V checked
    uint64_t pair[4];                          // the two softmax warps of 32 rows
    float pair_x[2][4][2][32];                 // what they exchange
    uint32_t tmem_base;
    int copies[2];    // bulk copies issued, for the drain
    volatile int abort;
    unsigned long long bad[kTreeMax / BK + 2];  // by tile of nodes: slots with a non-finite key or value
};

// A position in a ring of N slots: its index and the parity of its round.
template <int N>
struct Ring {
    int i = 0;
    unsigned ph = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) i = 0, ph ^= 1;
    }
};

template <typename S>
__device__ __forceinline__ bool twait(uint64_t* bar, unsigned parity, S& sm) {  // whole warp
    bool ok = false;
    for (unsigned i = 0; i < kWaitLimit && !ok; i++) {
        ok = mbar_try_wait(bar, parity);
        if (!ok && sm.abort) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) sm.abort = 1;
    return ok;
}
template <typename S>
__device__ __forceinline__ bool twait1(uint64_t* bar, unsigned parity, S& sm) {  // one thread
    for (unsigned i = 0; i < kWaitLimit; i++) {
        if (mbar_try_wait(bar, parity)) return true;
        if (sm.abort) return false;
    }
    sm.abort = 1;
    return false;
}

// Named barrier (whole warps), `threads` in all: some arrive, the others wait for them.
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_wait(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
// Whether the phase is complete, without waiting at all (a try_wait may suspend the warp for thousands of cycles).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, unsigned parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ float ex2u(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((unsigned)(min(max(e, -126), 127) + 127) << 23); }
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }  // x >= 0

// fp16 MN-major B operand: rows of 64 dims (128 B) per slot, 8-slot groups 1024 B apart, 64-dim chunks `chunk` apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t chunk) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)(chunk >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Whole warp: 16 columns of 32 lanes, waited for
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
// Whole warp: 16 columns of 32 lanes (waited for with tmem_st_wait)
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// The factor of scores, from q's and K's powers of two
__device__ __forceinline__ float score_factor(float qf, float kf) {
    return fminf(fmaxf(qf * kf, 0x1p-126f), 0x1p126f);  // (0 or inf times -inf or 0: NaN)
}

// x = hi + lo in fp16 (lo off by at most 2^-23 of x, or half of fp16's smallest step 2^-24)
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
    const __half2 a = __floats2half2_rn(x.x, x.y);
    const float2 r = fma2(__half22float2(a), both(-1.f), x);
    const __half2 b = __floats2half2_rn(r.x, r.y);
    hi = *reinterpret_cast<const uint32_t*>(&a);
    lo = *reinterpret_cast<const uint32_t*>(&b);
}

// ---------------------------------------------------------------- tiles of the converted cache types

// A lane's piece of its warp's 16 rows as they lie in the cache: piece i of a lane is piece i * 32 + lane of the rows in
// order, 16 bytes of fp32 values or 8 codes.
template <int TYPE>
struct Raw;
template <>
struct Raw<AF_F32> {
    static constexpr int VALUES = 4;
    uint4 a;
};
template <>
struct Raw<AF_KV_Q8_0> {
    static constexpr int VALUES = 8;
    uint2 a;
    __half d;
};
template <>
struct Raw<AF_KV_Q4_0> {
    static constexpr int VALUES = 8;
    uint32_t a;
    __half d;
};
template <int TYPE, int D>
constexpr int raw_pieces() {
    return 16 * D / Raw<TYPE>::VALUES / 32;
}
// A warp's rows in registers.  fp32 rows are kept from the look for their largest value to their conversion, so that the
// staging slot is free after the first (the slots hold less than two tiles of K and of V); codes are read again.
template <int TYPE, int D>
struct Kept {
    Raw<TYPE> c[TYPE == AF_F32 ? raw_pieces<TYPE, D>() : 1];
};

// Piece i from the staged rows st and their scales.  NODES: rows from `valid` on read as zeros, and so does what is not
// finite, whose rows are marked in `bad`.
template <int TYPE, int D, bool NODES>
__device__ __forceinline__ Raw<TYPE> load_raw(const uint8_t* st, const uint8_t* sc, int i, int valid, int lane, unsigned& bad) {
    const int idx = i * 32 + lane;
    Raw<TYPE> c;
    c.a = reinterpret_cast<const decltype(c.a)*>(st)[idx];
    if constexpr (TYPE != AF_F32) c.d = reinterpret_cast<const __half*>(sc)[idx / 4];
    if (NODES) {
        const int row = idx / (D / c.VALUES);
        if constexpr (TYPE == AF_F32) {
            uint32_t* w[4] = {&c.a.x, &c.a.y, &c.a.z, &c.a.w};
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (row >= valid || (*w[e] & 0x7F800000u) == 0x7F800000u) {
                    if (row < valid) bad |= 1u << row;
                    *w[e] = 0u;
                }
        } else {
            if (row >= valid || (__half_as_ushort(c.d) & 0x7C00u) == 0x7C00u) {
                if (row < valid) bad |= 1u << row;
                c.d = __ushort_as_half(0);
            }
        }
    }
    return c;
}

// The bits of the largest magnitude (or scale) of row `lane` of the warp's 16 (0 in the other lanes; NaNs count as above
// infinity).
template <int TYPE, int D, bool NODES>
__device__ __forceinline__ unsigned row_max(const uint8_t* st, const uint8_t* sc, int valid, int lane, unsigned& bad,
                                            Kept<TYPE, D>& kept) {
    unsigned mine = 0;
    if constexpr (TYPE == AF_F32) {
#pragma unroll
        for (int i = 0; i < raw_pieces<TYPE, D>(); i++) {  // one row a piece, or two (D = 64)
            const Raw<TYPE> c = load_raw<TYPE, D, NODES>(st, sc, i, valid, lane, bad);
            kept.c[i] = c;
            const unsigned m = max(max(c.a.x & 0x7FFFFFFFu, c.a.y & 0x7FFFFFFFu), max(c.a.z & 0x7FFFFFFFu, c.a.w & 0x7FFFFFFFu));
            if (D == 128) {
                const unsigned r = __reduce_max_sync(0xffffffffu, m);
                if (lane == i) mine = r;
            } else {
                const unsigned r0 = __reduce_max_sync(0xffffffffu, lane < 16 ? m : 0u);
                const unsigned r1 = __reduce_max_sync(0xffffffffu, lane < 16 ? 0u : m);
                if (lane >> 1 == i) mine = lane & 1 ? r1 : r0;
            }
        }
    } else if (lane < 16) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < D / 64; i++) {  // two scales
            unsigned w = reinterpret_cast<const unsigned*>(sc)[lane * (D / 64) + i] & 0x7FFF7FFFu;
            if (NODES) {
                const bool lo = (w & 0x7C00u) == 0x7C00u, hi = (w & 0x7C000000u) == 0x7C000000u;
                if (lane < valid && (lo || hi)) bad |= 1u << lane;
                w = lane < valid ? w & ((lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u)) : 0u;
            }
            m = max(m, max(w & 0xFFFFu, w >> 16));
        }
        mine = __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    }
    return mine;
}

// The exponents with which a warp's 16 rows are stored: row `lane`'s own one and the factor 2^-that (NaN: the row holds an
// infinity or a NaN, and every row of q sees it, since others are taken out: at its exponent the finite values would
// vanish).  Where they differ little, all rows have the largest.
struct RowExps {
    int e;       // of row `lane` (< 16); kNoExp: zeros
    float down;
    int hi;
    unsigned largest;  // bits of the largest value
    bool own;
    __device__ __forceinline__ float factor() const { return pow2i(hi); }
    __device__ __forceinline__ float exponent() const { return hi == kNoExp ? CUDART_NAN_F : (float)hi; }
};
template <int TYPE>
__device__ __forceinline__ RowExps row_exps(unsigned bits) {
    // largest value in [1, 2), or largest scale times its largest code in [1, 4)
    constexpr int code = TYPE == AF_KV_Q8_0 ? 6 : TYPE == AF_KV_Q4_0 ? 2 : 0;
    auto exponent = [](unsigned b) { return b ? min(max((int)(b >> 23) - 127, -126) + code, kMaxExp) : kNoExp; };
    RowExps x;
    x.largest = __reduce_max_sync(0xffffffffu, bits);
    x.hi = exponent(x.largest);
    const int e = exponent(bits);
    const bool inf = bits >= 0x7F800000u;
    x.own = __any_sync(0xffffffffu, inf || (e != kNoExp && e < x.hi - kSpread));
    x.e = x.own ? e : x.hi;
    x.down = inf ? CUDART_NAN_F : pow2i(-x.e);
    return x;
}

// Arrive, not before x (never all ones) has been computed.
__device__ __forceinline__ void mbar_arrive_after(uint64_t* bar, unsigned x) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0xffffffff;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(x)
        : "memory");
}

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// The fp16 hi and lo parts of the warp's rows row0.., times their 2^-exponent, into a slot (SWIZZLE_128B atoms of 64 dims,
// [64 slots][128 B] each).  fp32 rows with exponents of their own are read again by store_own (rare: rolled, and apart
// from the registers that keep the rows).
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int key, int d0) {
    return (uint32_t)((d0 >> 6) * BK * 128) + sw128(key, (d0 >> 3) & 7) + (d0 & 7) * 2;
}
template <int D>
__device__ __noinline__ void store_own(uint8_t* dst, const uint8_t* st, const RowExps& x, int row0, int valid, int lane) {
#pragma unroll 1
    for (int i = 0; i < raw_pieces<AF_F32, D>(); i++) {
        unsigned bad = 0;
        const Raw<AF_F32> r = load_raw<AF_F32, D, true>(st, nullptr, i, valid, lane, bad);  // (past: non-finite rows become NaN)
        const int idx = i * 32 + lane;
        const float2 dd = both(__shfl_sync(0xffffffffu, x.down, idx / (D / 4)));
        const uint32_t off = tile_offset<D>(row0 + idx / (D / 4), idx % (D / 4) * 4);
        uint2 hi, lo;
        split2(mul2(make_float2(__uint_as_float(r.a.x), __uint_as_float(r.a.y)), dd), hi.x, lo.x);
        split2(mul2(make_float2(__uint_as_float(r.a.z), __uint_as_float(r.a.w)), dd), hi.y, lo.y);
        *reinterpret_cast<uint2*>(dst + off) = hi;
        *reinterpret_cast<uint2*>(dst + BK * D * 2 + off) = lo;
    }
}
template <int TYPE, int D, bool NODES>
__device__ __forceinline__ void store_tile(uint8_t* dst, const uint8_t* st, const uint8_t* sc, const RowExps& x, int row0, int valid,
                                           int lane, const Kept<TYPE, D>& kept) {
    constexpr int PPR = D / Raw<TYPE>::VALUES, PART = BK * D * 2;  // pieces per row
    const float all = pow2i(-x.hi);
#pragma unroll
    for (int i = 0; i < raw_pieces<TYPE, D>(); i++) {
        unsigned bad = 0;
        const Raw<TYPE> r = TYPE == AF_F32 ? kept.c[TYPE == AF_F32 ? i : 0] : load_raw<TYPE, D, NODES>(st, sc, i, valid, lane, bad);
        const int idx = i * 32 + lane, key = row0 + idx / PPR, d0 = idx % PPR * Raw<TYPE>::VALUES;
        const uint32_t off = tile_offset<D>(key, d0);
        if constexpr (TYPE == AF_F32) {
            const uint4 a = r.a;
            const float2 dd = both(all);
            uint2 hi, lo;
            split2(mul2(make_float2(__uint_as_float(a.x), __uint_as_float(a.y)), dd), hi.x, lo.x);
            split2(mul2(make_float2(__uint_as_float(a.z), __uint_as_float(a.w)), dd), hi.y, lo.y);
            *reinterpret_cast<uint2*>(dst + off) = hi;
            *reinterpret_cast<uint2*>(dst + PART + off) = lo;
        } else {
            uint32_t hi[4], lo[4];
            // codes q are exact in fp16, and so is d 2^-e (11 bits); hi = fp16(q d), lo = q d - hi by a fused
            // multiply-add, exact as long as it is not below fp16's smallest step 2^-24
            const __half2 d2 = __float2half2_rn(__half2float(r.d) * __shfl_sync(0xffffffffu, x.down, idx / PPR));
            __half2 q[4];
            if constexpr (TYPE == AF_KV_Q8_0) {
                const uint32_t w = r.a.x ^ 0x80808080u, y = r.a.y ^ 0x80808080u;
                const __half2 off = u2h(0x64806480u);
                q[0] = __hsub2(u2h(__byte_perm(w, 0x64646464u, 0x4140)), off);
                q[1] = __hsub2(u2h(__byte_perm(w, 0x64646464u, 0x4342)), off);
                q[2] = __hsub2(u2h(__byte_perm(y, 0x64646464u, 0x4140)), off);
                q[3] = __hsub2(u2h(__byte_perm(y, 0x64646464u, 0x4342)), off);
            } else {
                const __half2 off = u2h(0x64086408u);
                const uint32_t w = r.a;
                __half2 n[4];  // dims (p, p + 4)
#pragma unroll
                for (int p = 0; p < 4; p++) n[p] = __hsub2(u2h(((w >> (4 * p)) & 0x000F000Fu) | 0x64006400u), off);
                q[0] = __lows2half2(n[0], n[1]);
                q[1] = __lows2half2(n[2], n[3]);
                q[2] = __highs2half2(n[0], n[1]);
                q[3] = __highs2half2(n[2], n[3]);
            }
#pragma unroll
            for (int p = 0; p < 4; p++) {
                const __half2 h = __hmul2_rn(q[p], d2);
                hi[p] = h2u(h);
                lo[p] = h2u(__hfma2(q[p], d2, __hneg2(h)));
            }
            *reinterpret_cast<uint4*>(dst + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(dst + PART + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// Half of a tile (32 slots a thread) where keys or values differ too much for one exponent in 16 or 64 slots.  Its scores in
// tensor memory become scores plus V's exponent (-infinity for zero values), so that the common code weighs them as if all
// exponents were 0; the largest score and the sum of 2^(score - that) come back.  Rare, and out of line: among the
// common tiles' code it cost them 3 to 8%.  (64 nodes over 30720 slots with every tile of this kind: fp32 210 us where
// others take 111, Q8_0 164 and 91.)
__device__ __noinline__ float2 own_scores(uint32_t s_addr, const int8_t* ek, const int8_t* ev, float rowf, unsigned see, unsigned bad) {
    float m = -CUDART_INF_F, l = 0.f;
    for (int c = 0; c < 32; c += 16) {
        float s[16];
        uint32_t u[16];
        tmem_ld16(s_addr + c, s);
#pragma unroll
        for (int i = 0; i < 16; i++) {
            s[i] *= score_factor(rowf, pow2i(ek[c + i]));
            if (bad >> (c + i) & 1) s[i] = CUDART_NAN_F;
            if (!(see >> (c + i) & 1)) s[i] = -CUDART_INF_F;
            m = fmaxf(m, s[i]);
            u[i] = __float_as_uint(s[i]);
        }
        tmem_st16(s_addr + c, u);
        tmem_st_wait();
    }
    const float m0 = m == -CUDART_INF_F ? 0.f : m;
    for (int c = 0; c < 32; c += 16) {
        float s[16];
        uint32_t u[16];
        tmem_ld16(s_addr + c, s);
#pragma unroll
        for (int i = 0; i < 16; i++) {
            l += ex2u(s[i] - m0);
            u[i] = __float_as_uint(s[i] + (ev[c + i] == kNoExp ? -CUDART_INF_F : (float)ev[c + i]));
        }
        tmem_st16(s_addr + c, u);
        tmem_st_wait();
    }
    return make_float2(m, l);
}

// ---------------------------------------------------------------- the kernel

template <int TYPE, int D>
__global__ void __launch_bounds__(TcCfgT<TYPE, D>::WARPS * 32, 1)
    attn_tree_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, TreeArgs a,
                        int tiles, int splits) {
    using C = TcCfgT<TYPE, D>;
    constexpr uint32_t kIdS = idesc_f16(kRows, BK);                  // scores: N = slots, B K-major
    constexpr uint32_t kIdO = idesc_f16(kRows, D) | (1u << 16);      // output: N = dims, B MN-major
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ TcState<C> sm;
    static_assert(sizeof(sm) + C::SMEM <= 227 * 1024, "an SM's shared memory");
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int G = a.H / a.c.KVH, R = a.n * G;
    const int split = blockIdx.x, g = blockIdx.y, r0 = blockIdx.z * kRows;
    const int t0 = (int)((int64_t)tiles * split / splits), T = (int)((int64_t)tiles * (split + 1) / splits) - t0;
    const int64_t row0 = (int64_t)g * a.c.ctx + (int64_t)t0 * BK;  // first slot row of the split
    // tiles from tn on hold nodes (or nothing behind them); slots from `valid` on, both counted from t0
    const int tn = a.past / BK - t0, valid = a.past + a.n - t0 * BK;

    if (tid == 0) {
        for (int x = 0; x < 2; x++) {
            for (int i = 0; i < C::NS; i++) {
                mbar_init(&sm.full[x][i], C::SPLIT ? kConvWarps : 1);
                mbar_init(&sm.empty[x][i], 1);
            }
            for (int i = 0; i < C::NR; i++) {
                mbar_init(&sm.raw_full[x][i], C::SCB ? 33 : 1);  // the copy's bytes, and each lane's scales
                mbar_init(&sm.raw_empty[x][i], kConvWarps);
            }
            sm.copies[x] = 0;
        }
        for (int i = 0; i < C::SB; i++) {
            mbar_init(&sm.s_full[i], C::SPLIT ? 2 : 1);  // the commit, and the issuer for K's exponent
            mbar_init(&sm.p_full[i], kSoftWarps);
            mbar_init(&sm.pv_done[i], 1);
        }
        for (int i = 0; i < 4; i++) mbar_init(&sm.pair[i], 2);
        mbar_init(&sm.v_clean, kSoftWarps);
        mbar_init(&sm.q_ready, kSoftWarps);
        mbar_init(&sm.done, 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < (int)(sizeof(sm.bad) / 8); i += C::WARPS * 32) sm.bad[i] = 0;
    if (warp == C::MMA_WARP) tmem_alloc(&sm.tmem_base, kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    // (softmax threads) where the thread's row of q starts
    const int qr = r0 + (warp & 3) * 32 + lane;
    const int64_t qoff = qr < R ? (int64_t)(qr / G) * a.ldq + (int64_t)(g * G + qr % G) * D : 0;
    // q and the output pass through the last V slots, so that global accesses are whole rows: chunk c (16 bytes) of row rr
    // of 32 sits at c ^ (rr & 7).
    constexpr int CPR = D / 4;  // chunks per row
    auto stage = [&](int quad, int rr, int c) {
        return reinterpret_cast<float4*>(smem + C::OFF_V + (C::NS - C::QS) * C::SLOT + (quad * 32 + rr) * D * 4 + ((c ^ (rr & 7)) << 4));
    };
    float row_l = 0.f, row_m = 0.f;  // (softmax threads) the row's sum, maximum and exponent
    float row_ev = 0.f;
    pdl_wait();  // q, the mask and the cache are written by earlier kernels

    if (warp == C::MMA_WARP) {
        // ---------------- MMA issuer: the whole warp walks the tiles (so that descriptors stay in uniform
        // registers), one elected lane issues
        const bool lead = elect_one();
        const uint32_t sbase = smem_u32(smem);
        const uint64_t kd0 = umma_desc_sw128(sbase), vd0 = desc_mn(sbase + C::OFF_V, BK * 128);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        constexpr int SB = C::SB;
        Ring<C::NS> rk, rv;
        bool ok = twait(&sm.q_ready, 0, sm);
        tc_fence_after();
        // here and not at the top: the next kernel's blocks start beside the first tiles, not beside q's loads (64 nodes
        // over 448 fp16 slots: 10.5 us, 11.0 from the top)
        pdl_launch_dependents();
        // A step's barriers are looked at while the previous step is being issued (the pipe is busy with it); only if
        // they were not all complete is there a wait.
        auto scores_ready = [&](int t) {
            return (t < SB || mbar_test(&sm.pv_done[t % SB], (t / SB - 1) & 1)) && mbar_test(&sm.full[0][rk.i], rk.ph);
        };
        auto scores_wait = [&](int t) {
            return (t < SB || twait(&sm.pv_done[t % SB], (t / SB - 1) & 1, sm)) && twait(&sm.full[0][rk.i], rk.ph, sm);
        };
        auto out_ready = [&](int t) {
            return mbar_test(&sm.full[1][rv.i], rv.ph) && mbar_test(&sm.p_full[t % SB], (t / SB) & 1);
        };
        auto out_wait = [&](int t) { return twait(&sm.full[1][rv.i], rv.ph, sm) && twait(&sm.p_full[t % SB], (t / SB) & 1, sm); };
        auto scores = [&](int t, int from, int to) {
            if (!lead) return;
            const uint64_t kd = kd0 + (uint32_t)(rk.i * (C::SLOT >> 4));
            const uint32_t d = tm + C::SCOL + t % SB * BK;
#pragma unroll
            for (int i = from; i < to; i++) {  // steps of lo products, then of hi products
                const int kk = i % (D / 16);
                const uint64_t b = kd + (((kk >> 2) * BK * 128 + (kk & 3) * 32) >> 4);
                if (i < D / 16) {
                    mma_f16_ts(d, tm + C::QCOL + D / 2 + kk * 8, b, kIdS, kk > 0);
                    if (C::SPLIT) mma_f16_ts(d, tm + C::QCOL + kk * 8, b + (C::PART >> 4), kIdS, 1);
                } else {
                    mma_f16_ts(d, tm + C::QCOL + kk * 8, b, kIdS, 1);
                }
            }
            if (to == D / 8) {
                mma_commit(&sm.s_full[t % SB]);
                mma_commit(&sm.empty[0][rk.i]);
                if (C::SPLIT) mbar_arrive(&sm.s_full[t % SB]);
            }
        };
        auto out = [&](int t, int from, int to) {
            if (!lead) return;
            const uint64_t vd = vd0 + (uint32_t)(rv.i * (C::SLOT >> 4));
            const uint32_t p = tm + C::SCOL + t % SB * BK;
#pragma unroll
            for (int i = from; i < to; i++) {
                const int kk = i % (BK / 16);
                const uint64_t b = vd + ((kk * 2048) >> 4);
                const uint32_t hi = p + (kk >> 1) * 32 + (kk & 1) * 8, lo = hi + 16;
                if (i < BK / 16) {
                    mma_f16_ts(tm, lo, b, kIdO, t % kFlush > 0 || kk > 0);
                    if (C::SPLIT) mma_f16_ts(tm, hi, b + (C::PART >> 4), kIdO, 1);
                } else {
                    mma_f16_ts(tm, hi, b, kIdO, 1);
                }
            }
            if (to == BK / 8) {
                mma_commit(&sm.pv_done[t % SB]);
                mma_commit(&sm.empty[1][rv.i]);
            }
        };
        for (int t = 0; ok && t < min(C::AHEAD, T); t++) {
            ok = scores_wait(t);
            if (!ok) break;
            tc_fence_after();
            scores(t, 0, D / 8);
            __syncwarp();
            rk.next();
        }
        bool next = false;  // the next step's barriers have been seen complete
        for (int t = 0; ok && t < T; t++) {
            const bool more = t + C::AHEAD < T;
            ok = next || out_wait(t);
            if (!ok) break;
            tc_fence_after();
            out(t, 0, BK / 8 - 2);
            __syncwarp();
            next = more && __all_sync(0xffffffffu, scores_ready(t + C::AHEAD));
            out(t, BK / 8 - 2, BK / 8);
            __syncwarp();
            rv.next();
            if (more) {
                ok = next || scores_wait(t + C::AHEAD);
                if (!ok) break;
                tc_fence_after();
                scores(t + C::AHEAD, 0, D / 8 - 4);
                __syncwarp();
                next = __all_sync(0xffffffffu, out_ready(t + 1));
                scores(t + C::AHEAD, D / 8 - 4, D / 8);
                __syncwarp();
                rk.next();
            } else {
                next = false;
            }
        }
        if (lead) mma_commit(&sm.done);  // always: the drain waits on it
    } else if (warp >= C::COPY_WARP) {
        const int x = warp - C::COPY_WARP;  // 0: K, 1: V
        bar_wait(kQueueBar, (kSoftWarps + 2) * 32);
        if constexpr (!C::SPLIT) {
            // ---------------- fp16: TMA straight into the operand layout
            if (lane == 0) {
                Ring<C::NS> r;
                for (int t = 0; t < T; t++, r.next()) {
                    if (t >= C::NS && !twait1(&sm.empty[x][r.i], r.ph ^ 1, sm)) break;
                    if (x == 1 && t == C::NS - C::QS && !twait1(&sm.q_ready, 0, sm)) break;
                    mbar_arrive_expect_tx(&sm.full[x][r.i], C::PART);
                    for (int d = 0; d < D; d += 64)
                        tma_load_2d(smem + (x ? C::OFF_V : 0) + r.i * C::SLOT + d * BK * 2, x ? &map_v : &map_k, d,
                                    (int)(row0 + t * BK), &sm.full[x][r.i]);
                    sm.copies[x] = t + 1;
                }
            }
        } else {
            // ---------------- raw rows into the staging ring: one bulk copy, and the scales by the lanes
            const uint8_t* src = (const uint8_t*)(x ? a.c.v : a.c.k) + row0 * C::RB;
            const uint8_t* sc = (const uint8_t*)(x ? a.c.vs : a.c.ks) + row0 * C::SCB;
            Ring<C::NR> r;
            // The scales go through registers, a slot ahead: copies of 4 or 8 bytes (rows may start off 16) would go
            // through L1, which may hold what an earlier kernel of the chain has overwritten since.
            constexpr int NS = C::SCB ? C::RR / 32 : 1;
            uint2 scale[NS] = {};
            auto fetch = [&](int i) {
                if (C::SCB == 0) return;
#pragma unroll
                for (int k = 0; k < NS; k++) {
                    const uint8_t* p = sc + ((int64_t)i * C::RR + k * 32 + lane) * C::SCB;
                    scale[k] = make_uint2(0u, 0u);
                    if (i * C::RR + k * 32 + lane < valid) {
                        if (C::SCB == 8)
                            scale[k] = __ldcg(reinterpret_cast<const uint2*>(p));
                        else
                            scale[k].x = __ldcg(reinterpret_cast<const unsigned*>(p));
                    }
                }
            };
            const int slots = T * (BK / C::RR);
            fetch(0);
            for (int i = 0; i < slots; i++, r.next()) {
                if (i >= C::NR && !twait(&sm.raw_empty[x][r.i], r.ph ^ 1, sm)) break;
                uint8_t* dst = smem + C::OFF_RAW + (x * C::NR + r.i) * C::RAW;
                const int rows = min(C::RR, max(0, valid - i * C::RR));
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sm.raw_full[x][r.i], rows * C::RB);
                    if (rows) bulk_g2s(dst, src + (int64_t)i * C::RR * C::RB, rows * C::RB, &sm.raw_full[x][r.i]);
                    sm.copies[x] = i + 1;
                }
                if (C::SCB) {
#pragma unroll
                    for (int k = 0; k < NS; k++) {
                        uint8_t* p = dst + C::RR * C::RB + (k * 32 + lane) * C::SCB;
                        if (C::SCB == 8)
                            *reinterpret_cast<uint2*>(p) = scale[k];
                        else
                            *reinterpret_cast<unsigned*>(p) = scale[k].x;
                    }
                    mbar_arrive(&sm.raw_full[x][r.i]);
                    if (i + 1 < slots) fetch(i + 1);
                }
            }
        }
    } else if (warp >= kSoftWarps) {
        if constexpr (C::SPLIT) {
            // ---------------- fp32, Q8_0, Q4_0: staged rows -> fp16 parts
            const int x = (warp - kSoftWarps) / kConvWarps, w = (warp - kSoftWarps) % kConvWarps;
            Ring<C::NR> rr;
            Ring<C::NS> ro;
            bool ok = true;
            for (int t = 0; t < T; t++, ro.next()) {
                // Every warp waits for every staging slot of the tile and frees it, the ones without its rows too: a
                // warp that skipped a round of a slot could not tell that round's completion from the next one's.
                // A slot is freed once its values have been used (fp32: their maximum depends on all of them; codes: after
                // they are stored): an arrival may overtake loads that are still queued, and the next copy then overwrites
                // what they read (seen as wrong results of single CTAs).
                int mine = 0;
#pragma unroll
                for (int p = 0; p < kConvWarps / C::RU; p++, rr.next()) {
                    ok = ok && twait(&sm.raw_full[x][rr.i], rr.ph, sm);
                    if (!ok) break;
                    if (w / C::RU == p)
                        mine = rr.i;
                    else if (lane == 0)
                        mbar_arrive(&sm.raw_empty[x][rr.i]);
                }
                if (!ok) break;
                const uint8_t* st = smem + C::OFF_RAW + (x * C::NR + mine) * C::RAW;
                const int wr = (w % C::RU) * 16;  // the warp's rows in the slot
                const uint8_t *rows = st + wr * C::RB, *scales = st + C::RR * C::RB + wr * C::SCB;
                const int left = t >= tn ? valid - t * BK - w * 16 : 16;  // the warp's rows that hold slots
                unsigned bad = 0, m;
                Kept<TYPE, D> kept;
                if (t >= tn)
                    m = row_max<TYPE, D, true>(rows, scales, left, lane, bad, kept);
                else
                    m = row_max<TYPE, D, false>(rows, scales, left, lane, bad, kept);
                const RowExps exps = row_exps<TYPE>(m);
                if (TYPE == AF_F32 && !exps.own && lane == 0) mbar_arrive_after(&sm.raw_empty[x][mine], exps.largest);
                if (bad) atomicOr(&sm.bad[t - tn], (unsigned long long)bad << (w * 16));
                if (t >= C::NS) ok = twait(&sm.empty[x][ro.i], ro.ph ^ 1, sm);
                if (x == 1 && t == C::NS - C::QS) ok = ok && twait(&sm.q_ready, 0, sm);
                if (!ok) break;
                uint8_t* dst = smem + (x ? C::OFF_V : 0) + ro.i * C::SLOT;
                if (TYPE == AF_F32 && exps.own)
                    store_own<D>(dst, rows, exps, w * 16, left, lane);
                else if (t >= tn)
                    store_tile<TYPE, D, true>(dst, rows, scales, exps, w * 16, left, lane, kept);
                else
                    store_tile<TYPE, D, false>(dst, rows, scales, exps, w * 16, left, lane, kept);
                if (lane < 16) (x ? sm.ev[ro.i] : sm.ek[t % C::EK])[w * 16 + lane] = (int8_t)exps.e;
                if (lane == 0) (x ? sm.vf[ro.i] : sm.kf[t % C::EK])[w] = exps.own ? CUDART_INF_F : x ? exps.exponent() : exps.factor();
                __syncwarp();
                if ((TYPE != AF_F32 || exps.own) && lane == 0) mbar_arrive(&sm.raw_empty[x][mine]);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.full[x][ro.i]);
            }
        }
    } else {
        // ---------------- softmax: thread = row and half of a tile's slots
        const int quad = warp & 3, half = warp >> 2;
        const int r = r0 + quad * 32 + lane;
        const bool live = r < R;
        const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
        unsigned pair_ph = 0;
        auto meet = [&]() {  // both warps of the rows
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.pair[quad]);
            const bool met = twait(&sm.pair[quad], pair_ph, sm);
            pair_ph ^= 1;
            return met;
        };
        float rowf = 1.f;
        constexpr int RPI = 32 / CPR;  // rows per warp access
        bool ok;
        {  // q: scaled to [1, 2), split, into tensor memory; each warp brings 16 rows and converts half of the dims
            const int c = lane % CPR, i0 = half * 16;
#pragma unroll
            for (int i = 0; i < 16 / RPI; i++) {
                const int rr = i0 + i * RPI + lane / CPR;
                const int64_t o = __shfl_sync(0xffffffffu, qoff, rr);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(stage(quad, rr, c))), "l"(a.q + o + c * 4) : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            bar_arrive(kQueueBar, (kSoftWarps + 2) * 32);  // K's and V's copies come after q, which is waited for first
            ok = meet();
            // half of the row's dims each; what a dead row reads may be anything
            float4 y[CPR / 2];
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < CPR / 2; i++) {
                y[i] = *stage(quad, lane, half * (CPR / 2) + i);
                mx = fmaxf(mx, fmaxf(fmaxf(fabsf(y[i].x), fabsf(y[i].y)), fmaxf(fabsf(y[i].z), fabsf(y[i].w))));
            }
            sm.pair_x[1][quad][half][lane] = mx;
            ok = ok && meet();
            mx = fmaxf(mx, sm.pair_x[1][quad][half ^ 1][lane]);
            const float sc = live ? rsqrtf((float)D) * 1.4426950408889634f : 0.f;
            const int e = min(max(exponent_of(mx * sc), -100), 126);
            rowf = pow2i(e);
            const float2 k = both(pow2i(-e)), scale = both(sc);
#pragma unroll
            for (int h = 0; h < D / 64; h++) {  // 32 dims: 16 columns of hi parts, 16 of lo parts
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float4 z = y[h * 8 + i];
                    split2(live ? mul2(mul2(make_float2(z.x, z.y), scale), k) : both(0.f), hi[2 * i], lo[2 * i]);
                    split2(live ? mul2(mul2(make_float2(z.z, z.w), scale), k) : both(0.f), hi[2 * i + 1], lo[2 * i + 1]);
                }
                const int col = (half * (D / 64) + h) * 16;
                tmem_st16(lane_addr + C::QCOL + col, hi);
                tmem_st16(lane_addr + C::QCOL + D / 2 + col, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            fence_proxy_async_shared();  // the slots may be filled
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_ready);
        }
        const int words = (a.n + 31) / 32;
        const unsigned* mrow = live ? a.mask + (int64_t)(r / G) * words : nullptr;
        auto window = [&](int t) {  // bit i: the row sees node t + i (t < 0: slots of the past, which every row sees)
            const int w = t >> 5;
            const unsigned lo = w < 0 ? ~0u : (mrow && w < words ? __ldcg(mrow + w) : 0u);
            const unsigned hi = w + 1 < 0 ? ~0u : (mrow && w + 1 < words ? __ldcg(mrow + w + 1) : 0u);
            const unsigned x = __funnelshift_r(lo, hi, t & 31);
            return t + 32 <= a.n ? x : (t >= a.n ? 0u : x & ((1u << (a.n - t)) - 1u));  // nothing behind the last node
        };
        constexpr int NG = C::SPLIT ? 2 : 1, W = 32 / NG;  // exponents of this half, slots of each
        float m_ref = -CUDART_INF_F, l = 0.f;
        // The output holds sums of w V 2^-ev, w = p 2^(ev - ev_ref): ev_ref keeps the largest score plus exponent of V so far
        // (z_run) near m_ref + ev_ref.
        float ev_ref = kNoRef, z_run = -CUDART_INF_F;
        Ring<C::NS> rv;
        for (int t = 0; ok && t < T; t++, rv.next()) {
            const int b = t % C::SB;
            const bool nodes = t >= tn;
            const unsigned see = nodes ? window((t0 + t) * BK - a.past + half * 32) : ~0u;
            ok = twait(&sm.s_full[b], (t / C::SB) & 1, sm);
            if (!ok) break;
            if (C::SPLIT || nodes) {
                ok = twait(&sm.full[1][rv.i], rv.ph, sm);  // V's exponents are there (K's since its scores were issued)
                if (!ok) break;
            }
            float f[NG], ev[NG], ev_hi = 0.f;
            bool apart = false;  // exponents differ too much for one in 16 (V: in 64) slots
#pragma unroll
            for (int q = 0; q < NG; q++) f[q] = rowf;
            if (C::SPLIT) {
                const float4 kf = *reinterpret_cast<const float4*>(sm.kf[t % C::EK]);
                const float4 vf = *reinterpret_cast<const float4*>(sm.vf[rv.i]);
                f[0] = score_factor(rowf, half ? kf.z : kf.x);
                f[NG - 1] = score_factor(rowf, half ? kf.w : kf.y);
                ev_hi = fmaxf(fmaxf(vf.x, vf.y), fmaxf(vf.z, vf.w));  // (not of zeros, NaN)
                const float ev_lo = fminf(fminf(vf.x, vf.y), fminf(vf.z, vf.w));
                apart = !(ev_hi - ev_lo <= (float)kSpread) || fmaxf(fmaxf(kf.x, kf.y), fmaxf(kf.z, kf.w)) == CUDART_INF_F;
                ev[0] = half ? vf.z : vf.x;
                ev[NG - 1] = half ? vf.w : vf.y;
            }
            if (!C::SPLIT && nodes) {  // V of this tile: zeros where it is not finite, and behind the last node
                uint8_t* v = smem + C::OFF_V + rv.i * C::SLOT;
#pragma unroll
                for (int i = 0; i < D / 32; i++) {
                    const int idx = i * kSoftWarps * 32 + tid, key = (idx >> 3) % BK;  // 16-byte chunk idx of [D / 64][64 slots][8]
                    uint4* p = reinterpret_cast<uint4*>(v) + idx;
                    uint4 x = *p;
                    uint32_t* w[4] = {&x.x, &x.y, &x.z, &x.w};
                    bool bad = false;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const bool lo = (*w[e] & 0x7C00u) == 0x7C00u, hi = (*w[e] & 0x7C000000u) == 0x7C000000u;
                        bad |= lo | hi;
                        *w[e] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
                    }
                    const bool out = t * BK + key >= valid;
                    if (out) x = make_uint4(0u, 0u, 0u, 0u);
                    if (bad || out) *p = x;
                    if (bad && !out) atomicOr(&sm.bad[t - tn], 1ull << key);
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.v_clean);
                ok = twait(&sm.v_clean, (t - max(tn, 0)) & 1, sm);
                if (!ok) break;
            }
            tc_fence_after();
            const uint32_t s_addr = lane_addr + C::SCOL + b * BK + half * 32;
            float own_m = 0.f, own_l = 0.f;
            if (C::SPLIT && apart) {  // (the same in every lane and in both warps of a row)
                const unsigned bad = nodes ? (unsigned)(*(volatile unsigned long long*)&sm.bad[t - tn] >> (half * 32)) : 0u;
                const float2 own = own_scores(s_addr, sm.ek[t % C::EK] + half * 32, sm.ev[rv.i] + half * 32, rowf, see, bad);
                sm.pair_x[t & 1][quad][half][lane] = own.x;
                ok = meet();
                own_m = fmaxf(own.x, sm.pair_x[t & 1][quad][half ^ 1][lane]);
                ok = ok && meet();  // (both have read it)
                if (!ok) break;
                own_l = own.x == -CUDART_INF_F ? own.y : own.y * ex2u(own.x - own_m);
#pragma unroll
                for (int q = 0; q < NG; q++) f[q] = 1.f, ev[q] = 0.f;
            }
            float s[32];
            tmem_ld32(s_addr, s);
            if (nodes) {
                const unsigned bad = (unsigned)(*(volatile unsigned long long*)&sm.bad[t - tn] >> (half * 32));
#pragma unroll
                for (int i = 0; i < 32; i++) {
                    if (bad >> i & 1) s[i] = CUDART_NAN_F;
                    if (!(see >> i & 1)) s[i] = -CUDART_INF_F;
                }
            }
            float mt = -CUDART_INF_F;
#pragma unroll
            for (int q = 0; q < NG; q++) {
                float x0 = s[q * W], x1 = s[q * W + 1];
#pragma unroll
                for (int i = 2; i < W; i += 4) {
                    x0 = fmaxf(fmaxf(x0, s[q * W + i]), s[q * W + i + 1]);
                    if (i + 2 < W) x1 = fmaxf(fmaxf(x1, s[q * W + i + 2]), s[q * W + i + 3]);
                }
                mt = fmaxf(mt, fmaxf(x0, x1) * f[q]);
            }
            sm.pair_x[t & 1][quad][half][lane] = mt;
            ok = meet();
            if (!ok) break;
            mt = fmaxf(mt, sm.pair_x[t & 1][quad][half ^ 1][lane]);
            const float z = C::SPLIT && apart ? mt : mt + ev_hi;  // the largest score plus exponent of V
            if (C::SPLIT && apart) mt = own_m;
            z_run = fmaxf(z_run, z);
            const bool move = mt > m_ref + kLazy2;
            const bool grow = C::SPLIT && z > m_ref + ev_ref + kLazy2;
            const bool flush = t > 0 && t % kFlush == 0;  // the output sum starts again with this tile
            const bool change = __any_sync(0xffffffffu, move || grow);  // (the same in both warps)
            if (change || flush) {
                float up = 1.f;
                if (change) {
                    float d = 0.f;
                    if (mt > m_ref) {
                        d = m_ref - mt;
                        m_ref = mt;
                        l *= ex2u(d);
                    }
                    if (C::SPLIT && z_run > -CUDART_INF_F) {
                        const float e = ceilf(fminf(fmaxf(z_run - m_ref, -126.f), 127.f));
                        d += ev_ref - e;
                        ev_ref = e;
                    }
                    up = ex2u(d);
                }
                if (t > 0) {  // the output holds the tiles before t: wait for them; half of the dims each
                    ok = twait(&sm.pv_done[(t - 1) % C::SB], ((t - 1) / C::SB) & 1, sm);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
                        float o[16], acc[16];
                        uint32_t u[16];
                        if (t > kFlush) tmem_ld16(lane_addr + C::ACC + c, acc);
                        tmem_ld16(lane_addr + c, o);
                        if (flush) {
#pragma unroll
                            for (int i = 0; i < 16; i++) u[i] = __float_as_uint((t > kFlush ? acc[i] + o[i] : o[i]) * up);
                            tmem_st16(lane_addr + C::ACC + c, u);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; i++) u[i] = __float_as_uint(o[i] * up);
                            tmem_st16(lane_addr + c, u);
                            if (t > kFlush) {
#pragma unroll
                                for (int i = 0; i < 16; i++) u[i] = __float_as_uint(acc[i] * up);
                                tmem_st16(lane_addr + C::ACC + c, u);
                            }
                        }
                    }
                    tmem_st_wait();
                }
            }
            const float mb = (m_ref == -CUDART_INF_F ? 0.f : m_ref) - kBias2;
            uint32_t p32[32];  // hi parts, then lo parts
#pragma unroll
            for (int q = 0; q < NG; q++) {
                // V's slots are 2^-ev of themselves and the output 2^-ev_ref: p takes the difference
                const float shift = C::SPLIT ? fmaxf(ev[q] - ev_ref, kNoRef) : 0.f;  // (zeros: NaN)
                const float2 ff = both(f[q]), mm = both(shift - mb);
                float2 sum[2] = {};
#pragma unroll
                for (int i = 0; i < W; i += 2) {
                    const float2 y = fma2(make_float2(s[q * W + i], s[q * W + i + 1]), ff, mm);
                    const float2 p = make_float2(ex2u(y.x), ex2u(y.y));
                    sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], p);
                    split2(p, p32[(q * W + i) / 2], p32[16 + (q * W + i) / 2]);
                }
                const float2 add = add2(sum[0], sum[1]);
                if (C::SPLIT && apart) {
                    if (q == 0) l += own_l * ex2u(own_m - mb);
                } else if (C::SPLIT && shift < -8.f) {  // small values: p's sum apart from their factor
                    float z = 0.f;
#pragma unroll
                    for (int i = 0; i < W; i++) z += ex2u(s[q * W + i] * f[q] - mb);
                    l += z;
                } else {
                    l += C::SPLIT ? (add.x + add.y) * ex2u(-shift) : add.x + add.y;
                }
            }
            tmem_st32(s_addr, p32);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[b]);
        }
        // ---- the row's sum is that of both halves
        if (ok) {
            sm.pair_x[T & 1][quad][half][lane] = l;
            ok = meet() && twait(&sm.done, 0, sm);
            l += sm.pair_x[T & 1][quad][half ^ 1][lane];
        }
        row_l = l;
        row_m = m_ref;
        row_ev = ev_ref;
    }
    tc_fence_before();
    __syncthreads();  // every wait is behind: whether one of them gave up holds for the whole CTA
    const bool gave_up = sm.abort;
    if (warp < kSoftWarps) {
        // ---------------- this split's part of the rows, half of the dims a thread
        const int quad = warp & 3, half = warp >> 2, r = r0 + quad * 32 + lane;
        const bool live = r < R, last = splits == 1;  // last: the result itself (zeros for a row that saw nothing)
        const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
        const int64_t rows = (int64_t)a.c.KVH * R;
        const int64_t row = (int64_t)split * rows + (int64_t)g * R + r;
        float* base = last ? a.out : a.ws;
        const int64_t off = !live ? 0 : last ? (int64_t)(r / G) * a.ldo + (int64_t)(g * G + r % G) * D : row * D;
        if (!gave_up) {  // every operand has been read: the ring is free
            constexpr int HC = CPR / 2;  // chunks of half a row
            tc_fence_after();
            float up = C::SPLIT ? pow2i((int)row_ev) : 1.f;
            if (last) up *= live ? row_inverse(a, r / G, row_l) : 0.f;
#pragma unroll 1
            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
                float o[32];
                tmem_ld32(lane_addr + c, o);
                if (T > kFlush) {
                    float acc[32];
                    tmem_ld32(lane_addr + C::ACC + c, acc);
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] += acc[i];
                }
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *stage(quad, lane, (c + i) / 4) = make_float4(o[i] * up, o[i + 1] * up, o[i + 2] * up, o[i + 3] * up);
            }
            __syncwarp();
            const int c = half * HC + lane % HC;
            int64_t o[HC];
#pragma unroll
            for (int i = 0; i < HC; i++) o[i] = __shfl_sync(0xffffffffu, off, i * (32 / HC) + lane / HC);
#pragma unroll
            for (int i = 0; i < HC; i++) {
                const int rr = i * (32 / HC) + lane / HC;
                if (r0 + quad * 32 + rr < R) reinterpret_cast<float4*>(base + o[i])[c] = *stage(quad, rr, c);
            }
        } else if (live) {  // copies and MMAs may still be in flight: nothing goes through shared memory
            for (int i = 0; i < D / 8; i++)
                reinterpret_cast<float4*>(base + off)[half * (D / 8) + i] =
                    make_float4(CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F);
        }
        if (live && !last && half == 0)
            reinterpret_cast<float2*>(a.ws + splits * rows * D)[row] =
                gave_up ? make_float2(CUDART_NAN_F, CUDART_NAN_F) : make_float2(row_m, row_l);
    }
    tc_fence_before();
    __syncthreads();
    if (gave_up && tid == 0) {  // let what was issued finish before leaving
        mbar_wait_bounded(&sm.done, 0);
        for (int x = 0; x < 2; x++) {
            constexpr int N = C::SPLIT ? C::NR : C::NS;
            for (int i = max(0, sm.copies[x] - N); i < sm.copies[x]; i++)
                mbar_wait_bounded(C::SPLIT ? &sm.raw_full[x][i % N] : &sm.full[x][i % N], (i / N) & 1);
        }
    }
    __syncthreads();
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_free(tmem, kTmem);
    }
}

template <int TYPE, int D>
cudaError_t go(const TreeArgs& a, const TreeTcPlan& p, cudaStream_t s) {
    using C = TcCfgT<TYPE, D>;
    auto k = attn_tree_tc_kernel<TYPE, D>;
    static SmemOptIn opt;
    cudaError_t e = opt((const void*)k, C::SMEM);
    if (e) return e;
    CUtensorMap mk = {}, mv = {};
    if (TYPE == AF_F16) {
        const uint64_t rows = (uint64_t)a.c.KVH * a.c.ctx;
        if (!make_tmap_f16(&mk, a.c.k, rows, D, D, 64, BK) || !make_tmap_f16(&mv, a.c.v, rows, D, D, 64, BK))
            return cudaErrorInvalidValue;
    }
    const int R = a.n * (a.H / a.c.KVH);
    return launch_chained(k, dim3(p.splits, a.c.KVH, (R + kRows - 1) / kRows), C::WARPS * 32, C::SMEM, s, mk, mv, a, p.tiles,
                          p.splits);
}

template <int TYPE>
cudaError_t go_type(const TreeArgs& a, const TreeTcPlan& p, cudaStream_t s) {
    return a.c.D == 64 ? go<TYPE, 64>(a, p, s) : go<TYPE, 128>(a, p, s);
}

}  // namespace

TreeTcPlan tree_tc_plan(int H, int KVH, int D, int type, int past, int n) {
    TreeTcPlan p;
    const int R = n * (H / KVH);
    // More than 32 rows; of fp32 caches, whose mma.sync kernel needs three tf32 products, more than 16 over a long past and
    // more than 8 over a longer one.  32 rows x 128 over fp32 slots, there and here: 1100 slots 13.9 and 14.6 us, 2000 20.0
    // and 17.4, 30000 108 and 62; x 64: 4000 15.6 and 19.6, 8192 22.1 and 23.8, 30000 63.8 and 48.6.  16 rows x 128: 4000
    // 16.5 and 22.9, 20400 49.6 and 47.7, 30000 67.0 and 61.9; x 64: 30000 34.4 and 49.0.  32 rows x 128 of the other types:
    // 4000 fp16 slots 14.1 and 17.4, 30000 38.1 and 39.0, 60000 62.0 and 61.2; 30000 Q8_0 42.6 and 51.5, Q4_0 40.5 and 51.1.
    int most = 32;
    if (type == AF_F32 && past + n >= (D == 128 ? 1536 : 8192)) most = D == 128 && past + n >= 20480 ? 8 : 16;
    if (R <= most) return p;
    p.tiles = (past + n + BK - 1) / BK;
    const int64_t ctas = (int64_t)KVH * ((R + kRows - 1) / kRows);
    // one CTA per SM, two tiles each or more (64 nodes over 448 fp16 slots: 10.6 us, 12.3 with four), but a few tiles are
    // not worth a merge (64 nodes over 192 slots: fp16 10.1 us in one split, 10.2 in two; fp32 14.2 and 13.0, Q8_0 12.5 and
    // 11.7)
    p.splits = p.tiles <= 4 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(num_sms() / ctas, p.tiles / 2));
    return p;
}

cudaError_t launch_attn_tree_tc(const TreeArgs& a, const TreeTcPlan& p, cudaStream_t s) {
    switch (a.c.type) {
        case AF_F32: return go_type<AF_F32>(a, p, s);
        case AF_F16: return go_type<AF_F16>(a, p, s);
        case AF_KV_Q8_0: return go_type<AF_KV_Q8_0>(a, p, s);
        default: return go_type<AF_KV_Q4_0>(a, p, s);
    }
}

}  // namespace af

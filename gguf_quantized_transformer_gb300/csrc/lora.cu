// Low-rank adapters of many requests beside a shared projection: row i of the batch with adapter a,
//   y_i = base_i + scale_a B_a (A_a x_i),   A_a [rank, K], B_a [N, rank].
//
// The rows are put in the order of their adapters once a step (lora_plan_kernel: a counting sort), in tiles of up to 32 rows
// of one adapter, so that an adapter's weights are read once for all of them.  Then two kernels:
//  - shrink: h = A x.  A CTA takes a tile, 16 or 32 ranks and a range of K, its warps chunks of 32 of that range in turn, each
//    through a ring of its own (lane c of 4 owns 8 values of a chunk, on both sides, so the order within it is free).  The
//    warps' sums join in shared memory, the ranges' sums by their reader, both in order.
//  - expand: y = base + B (scale h).  A CTA takes runs of 128 columns of one tile after another; h's parts lie in shared memory as
//    operands, a warp's 16 columns of B and their part of the base come through its ring, y is written in 16-byte pieces.
// Bound by the bytes of base, y and x for many rows of low rank (2048 rows of 5 fp16 adapters of rank 32 beside 4096 -> 28672 97 us,
// 5.3 TB/s), by two rounds of loads and a join in each kernel for few (one row of rank 16 beside 4096 -> 4096 4.9 us; 40 rows of
// 12 fp32 adapters of ranks 16 to 64 beside 14336 -> 4096 17.6 us for 39 MB; 64 rows of 40 of rank 16 beside 4096 -> 6144 12.6 us,
// in expand by its instructions: runs of 16 columns a warp for one or two rows).  Many rows of high rank or fp32 weights are bound
// by the weights, which are fetched from L2 and split again for every 32 rows (512 rows of one fp16 adapter of rank 128 beside
// 4096 -> 14336 37 us, 10.6 of them bytes; 2048 rows of 5 fp32 adapters of rank 64 beside 14336 -> 4096 100 us, 31 of them).
// Expand starts while shrink runs: what shrink does not write (the plan, B, the base) is fetched before its wait.  (All figures
// here and below are of calls in a graph.)
// Precision: fp16 products of two parts of 11 bits (x, h and fp32 weights; fp16 weights are operands as they are), after a power
// of two has brought the largest of a row's 32 values (of a chunk; of h all) to [2^13, 2^14), or [2^13, 2^15] with fp32 weights:
// 2^-22 of a value or half of fp16's smallest step of 2^-24, which is 2^-38 of the largest, stays.  The product of two low parts
// is left out.  Tensor cores cut their sums: those of a chunk start from zero, small products first, and are added in fp32.  (tf32
// needs no scaling, but mma.sync does 128 of its multiplications a cycle and SM.)
#include <algorithm>
#include <type_traits>

#include "mma_sync.cuh"
#include "serve.cuh"
#include "tma.cuh"

namespace af {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kThreads = 256, kWarps = kThreads / 32;  // of expand
// Warps of a CTA of shrink and the bytes of a warp's ring.  (fp16 of rank 16: as little shared memory as lets expand's CTAs in
// beside it: one row, 4096 -> 4096, 4.8 us; with 12 warps of 16 KB 5.6.  Higher ranks: as much as there is, 2048 rows of fp32
// adapters of rank 64 100 us, with 8 warps 104; 64 rows of 4 fp16 adapters of rank 64 go the other way, 17.1 and 16.0.)
template <bool F16, int MT>
constexpr int kShrinkWarps = F16 && MT == 1 ? 8 : 12;
template <bool F16, int MT>
constexpr int kRing = (F16 && MT == 1 ? 10 : 16) * 1024;
constexpr int kMaxSplit = 16;
constexpr int kHalf = 112 * 1024;  // shared memory of a CTA of expand that shares its SM with another
constexpr int kCols = 16 * kWarps;  // columns that a CTA of expand takes at once

__host__ __device__ inline int64_t plan_order(int max_tiles) { return 4 * (int64_t)(1 + max_tiles); }  // in ints

// ---------------------------------------------------------------- plan

constexpr int kTileBits = 14;  // rows and tiles are summed in one word: 18 bits of rows, 14 of tiles
constexpr unsigned kTileMask = (1u << kTileBits) - 1;
static_assert(kLoraMaxRows / kLoraTile + kLoraMaxAdapters + 1 <= (int)kTileMask && kLoraMaxRows < 1 << (32 - kTileBits), "");

__device__ __forceinline__ unsigned cta_scan(unsigned x, unsigned& total) {  // inclusive
    __shared__ unsigned part[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    const unsigned y = part[lane];
    total = __reduce_add_sync(0xffffffffu, y);
    return x + __reduce_add_sync(0xffffffffu, lane < warp ? y : 0u);
}

__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(const int* __restrict__ ids, int n, int adapters, int max_tiles,
                                                                  int* __restrict__ plan) {
    __shared__ int count[kLoraMaxAdapters + 1], first[kLoraMaxAdapters + 2];  // rows of an adapter; its first tile
    const int t = threadIdx.x, lane = t & 31;
    pdl_launch_dependents();
    pdl_wait();
    // a row's adapter; those without one count as the last, -1 behind the last row
    auto bucket = [&](int i) {
        const int id = i < n ? __ldcg(ids + i) : 0;
        return i >= n ? -1 : id >= 0 && id < adapters ? id : adapters;
    };
    const int mine = bucket(t);
    for (int i = t; i <= adapters; i += kPlanThreads) count[i] = 0;
    __syncthreads();
    // rows of each adapter, a warp's equal ones at once
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int b = i0 ? bucket(i0 + t) : mine;
        const unsigned same = __match_any_sync(0xffffffffu, b);
        if (b >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[b], __popc(same));
    }
    __syncthreads();
    int rows = 0, tiles = 0;
    const int bare = count[adapters];
    for (int i0 = 0; i0 <= adapters; i0 += kPlanThreads) {
        const int i = i0 + t, c = i <= adapters ? count[i] : 0, k = (c + kLoraTile - 1) / kLoraTile;
        unsigned total;
        const unsigned both = cta_scan((unsigned)c << kTileBits | (unsigned)k, total);
        if (i <= adapters) count[i] = rows + (int)(both >> kTileBits) - c, first[i] = tiles + (int)(both & kTileMask) - k;
        rows += (int)(total >> kTileBits);
        tiles += (int)(total & kTileMask);
    }
    if (t == 0) {
        first[adapters + 1] = tiles;
        const int bare_tiles = (bare + kLoraTile - 1) / kLoraTile;
        *reinterpret_cast<int4*>(plan) = make_int4(tiles, tiles - bare_tiles, n - bare, lora_plan_sizes(n, adapters));
    }
    __syncthreads();
    for (int i = t; i < tiles; i += kPlanThreads) {
        int lo = 0, hi = adapters + 1;  // first[lo] <= i < first[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        const int at = count[lo] + (i - first[lo]) * kLoraTile, end = lo == adapters ? n : count[lo + 1];
        reinterpret_cast<int4*>(plan)[1 + i] = make_int4(lo == adapters ? -1 : lo, at, min(kLoraTile, end - at), 0);
    }
    __syncthreads();
    int* const order = plan + plan_order(max_tiles);
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + t, b = i0 ? bucket(i) : mine;
        const unsigned same = __match_any_sync(0xffffffffu, b);
        const int lead = __ffs(same) - 1;
        int at = 0;
        if (b >= 0 && lane == lead) at = atomicAdd(&count[b], __popc(same));
        at = __shfl_sync(0xffffffffu, at, lead);
        if (b >= 0) order[at + __popc(same & ((1u << lane) - 1))] = i;
    }
}

// ---------------------------------------------------------------- rings

// 16 bytes through L2 into a shared-memory ring, of which the first `bytes` are read and the others zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// Tile i; the first 32, a lane each, come with the header
__device__ __forceinline__ int4 first_tiles(const int* plan, int lane, int max_tiles) {
    return __ldcg(reinterpret_cast<const int4*>(plan) + 1 + min(lane, max_tiles - 1));
}
__device__ __forceinline__ int4 tile_of(const int* plan, int i, const int4& early) {
    if (i >= 32) return __ldcg(reinterpret_cast<const int4*>(plan) + 1 + i);
    return make_int4(__shfl_sync(0xffffffffu, early.x, i), __shfl_sync(0xffffffffu, early.y, i), __shfl_sync(0xffffffffu, early.z, i), 0);
}

__device__ __forceinline__ int rank_of(const LoraArgs& a, int adapter) {
    return a.ranks ? min(max(__ldcg(a.ranks + adapter), 0), a.rank) : a.rank;
}

// ---------------------------------------------------------------- shrink

// Ranges of K: as many as every SM takes one of at once, of at least two chunks of 32 for each warp (64 rows of 4 fp16
// adapters of rank 64 beside 4096 -> 28672: 17.1 us; with three 18.2, with one, more to add up in expand, 18.1; one row 4.8, 5.3
// and 5.1)
__device__ __forceinline__ int lora_splits(int items, int K, int sms, int warps) {
    return max(1, min(min(sms / max(items, 1), kMaxSplit), K / 32 / (2 * warps)));
}


// 2^k that brings a largest magnitude m to [2^13, 2^14), and 2^-k.  (Below 2^-112 it comes no nearer.  An infinity stays one, and
// its low part is NaN: what it meets is NaN.)
__device__ __forceinline__ void powers(float m, float& down, float& up) {
    int e = (int)(__float_as_uint(m) >> 23) - 127;
    e = min(max(e, -112), 127);
    down = __uint_as_float((unsigned)(127 + 13 - e) << 23);
    up = __uint_as_float((unsigned)(127 - 13 + e) << 23);
}
// The same for fp32 weights and what meets them, for m >= kLeast: 2^k with k even brings it to [2^13, 2^15]; and 2^(-k / 2).  A sum
// of products is taken back by the product of two such roots, twice: that product is in [2^-126, 2^114], so that nothing on the
// way leaves fp32's range where the result does not.  (The sum times the weights' whole power alone is infinite for weights of
// 1e36, though x of 1e-36 brings it back.)
constexpr float kLeast = 0x1p-112f;
__device__ __forceinline__ void power_root(float m, float& down, float& root) {
    const int k = (int)(0x47000000u - __float_as_uint(m)) & ~0xFFFFFF;  // k 2^23: 15 less the exponent, the mantissa too, down to even
    down = __int_as_float(0x3F800000 + k);
    root = __int_as_float(0x3F800000 - (k >> 1));
}
// s p^2 + acc
__device__ __forceinline__ float2 back_from(const float2& s, const float2& p, const float2& acc) { return fma2(mul2(s, p), p, acc); }
// 8 values of lanes c = 0..3 (32 of one row) as scaled parts, in pairs; the power, or its ROOT, that takes the sums back
template <bool ROOT>
__device__ __forceinline__ float parts8(const uint4& v, const uint4& w, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    float x[8] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w),
                  __uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
    float m = ROOT ? kLeast : 0.f, down, up;
#pragma unroll
    for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(x[i]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (ROOT)
        power_root(m, down, up);
    else
        powers(m, down, up);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 y = mul2(make_float2(x[2 * i], x[2 * i + 1]), both(down));
        split_h2(y.x, y.y, hi[i], lo[i]);
    }
    return up;
}

// The sums of chunks k0 + warp, + NW .. below k1 for 16 MT ranks and 8 NT rows, in `sum`: [warps][16 MT][pad].
// Weights and x go through the warp's ring, whole lines of 128 bytes a row (64 of fp16 weights); in it odd rows have
// neighbouring 16-byte pieces exchanged, so that the reads meet all banks.
// w: the adapter's weights from the tile's first rank on; in: the ranks that there are from it on.
template <bool F16, int MT, int NT>
__device__ __forceinline__ void shrink_tile(const LoraArgs& a, const int* row, int count, const uint8_t* w, int in, int k0, int k1,
                                            uint32_t ring, float* sum, int pad) {
    constexpr int WB = 16 * MT * (F16 ? 64 : 128), STAGE = WB + 8 * NT * 128, NST = kRing<F16, MT> / STAGE < 8 ? kRing<F16, MT> / STAGE : 8, NW = kShrinkWarps<F16, MT>;
    static_assert(NST >= 2, "a stage in flight while one is read");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, j = lane >> 2, q = lane >> 3, e16 = lane & 7;
    auto fetch = [&](int k, int slot) {
        const uint32_t dst = ring + slot * STAGE;
        if constexpr (F16) {
#pragma unroll
            for (int i = 0; i < 2 * MT; i++) {
                const bool is = 8 * i + j < in;
                copy16(dst + i * 512 + lane * 16, is ? w + ((int64_t)(8 * i + j) * a.K + 32 * k + 8 * c) * 2 : (const uint8_t*)a.a, is ? 16 : 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4 * MT; i++) {
                const bool is = 4 * i + q < in;
                copy16(dst + (4 * i + q) * 128 + ((e16 ^ (q & 1)) << 4),
                       is ? w + ((int64_t)(4 * i + q) * a.K + 32 * k + 4 * e16) * 4 : (const uint8_t*)a.a, is ? 16 : 0);
            }
        }
#pragma unroll
        for (int i = 0; i < 2 * NT; i++) {
            const int r = 4 * i + q;
            const float* p = a.x + (r < count ? (int64_t)row[r] * a.ldx : 0) + 32 * k + 4 * e16;
            copy16(dst + WB + r * 128 + ((e16 ^ (q & 1)) << 4), p, r < count ? 16 : 0);
        }
    };
    // half h of the 8 values of row j of eight that lie in lines of 128 bytes
    auto line8 = [&](uint32_t at, int h) { return shared16(at + j * 128 + (((2 * c + h) ^ (j & 1)) << 4)); };
    float acc[MT][NT][4] = {};
    int ahead = k0 + warp;
#pragma unroll 1
    for (int i = 0; i < NST; i++, ahead += NW) {
        if (ahead < k1) fetch(ahead, i);
        copy_commit();
    }
    int slot = 0;
#pragma unroll 1
    for (int k = k0 + warp; k < k1; k += NW, ahead += NW) {
        copy_wait<NST - 1>();
        __syncwarp();  // the other lanes' pieces have landed
        const uint32_t at = ring + slot * STAGE;
        uint32_t xh[NT][4], xl[NT][4];
        float2 up[NT];  // of rows 2c and 2c + 1 of each 8 (fp32 weights: its root)
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const float u = parts8<!F16>(line8(at + WB + 1024 * t, 0), line8(at + WB + 1024 * t, 1), xh[t], xl[t]);
            up[t] = make_float2(__shfl_sync(0xffffffffu, u, 8 * c), __shfl_sync(0xffffffffu, u, 8 * c + 4));
        }
#pragma unroll
        for (int m = 0; m < MT; m++) {
            uint32_t hi[2][4], lo[2][4];
            float wup[2] = {1.f, 1.f};
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if constexpr (F16) {
                    const uint4 v = shared16(at + (2 * m + h) * 512 + lane * 16);
                    hi[h][0] = v.x, hi[h][1] = v.y, hi[h][2] = v.z, hi[h][3] = v.w;
                } else {
                    wup[h] = parts8<true>(line8(at + 1024 * (2 * m + h), 0), line8(at + 1024 * (2 * m + h), 1), hi[h], lo[h]);
                }
            }
            float s[NT][4];
#pragma unroll
            for (int t = 0; t < NT; t++) dot16z(s[t], make_uint4(hi[0][0], hi[1][0], hi[0][1], hi[1][1]), xl[t][0], xl[t][1]);
#pragma unroll
            for (int t = 0; t < NT; t++) dot16(s[t], make_uint4(hi[0][2], hi[1][2], hi[0][3], hi[1][3]), xl[t][2], xl[t][3]);
            if constexpr (!F16) {
#pragma unroll
                for (int e = 0; e < 4; e += 2)
#pragma unroll
                    for (int t = 0; t < NT; t++)
                        dot16(s[t], make_uint4(lo[0][e], lo[1][e], lo[0][e + 1], lo[1][e + 1]), xh[t][e], xh[t][e + 1]);
            }
#pragma unroll
            for (int e = 0; e < 4; e += 2)
#pragma unroll
                for (int t = 0; t < NT; t++) dot16(s[t], make_uint4(hi[0][e], hi[1][e], hi[0][e + 1], hi[1][e + 1]), xh[t][e], xh[t][e + 1]);
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float2 v = make_float2(s[t][2 * h], s[t][2 * h + 1]), z = make_float2(acc[m][t][2 * h], acc[m][t][2 * h + 1]);
                    const float2 y = F16 ? fma2(v, up[t], z) : back_from(v, mul2(up[t], both(wup[h])), z);
                    acc[m][t][2 * h] = y.x, acc[m][t][2 * h + 1] = y.y;
                }
        }
        __syncwarp();
        if (ahead < k1) fetch(ahead, slot);
        copy_commit();
        slot = slot + 1 == NST ? 0 : slot + 1;
    }
    copy_wait<0>();
    __syncthreads();  // (the sums take the rings' place)
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                *reinterpret_cast<float2*>(sum + (warp * 16 * MT + 16 * m + 8 * h + j) * pad + 8 * t + 2 * c) =
                    make_float2(acc[m][t][2 * h], acc[m][t][2 * h + 1]);
}

template <bool F16, int MT>
__global__ void __launch_bounds__(kShrinkWarps<F16, MT> * 32, 1) lora_shrink_kernel(LoraArgs a, int max_tiles, int sms) {
    constexpr int NW = kShrinkWarps<F16, MT>, RING = kRing<F16, MT>, RR = 16 * MT, PAD = kLoraTile + 2, es = F16 ? 2 : 4;
    static_assert(RR * PAD * 4 <= RING, "the sums fit the rings");
    extern __shared__ __align__(16) float sm_sum[];  // the warps' rings, then [warps][RR][PAD]
    __shared__ int sm_row[kLoraTile], sm_order[NW * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int* plan = (const int*)a.plan;
    pdl_wait();
    pdl_launch_dependents();  // (behind the wait: expand reads what is older than this kernel before its own)
    const int* const order = plan + plan_order(max_tiles);
    const int early_row = tid < a.n ? __ldcg(order + tid) : 0;
    const int4 head = __ldcg(reinterpret_cast<const int4*>(plan));
    const int4 early = first_tiles(plan, lane, max_tiles);
    const int tiles = head.w == lora_plan_sizes(a.n, a.adapters) ? head.y : 0;  // (another call's plan: nothing, see expand)
    const int rows = head.z, rt = (a.rank + RR - 1) / RR;
    const int splits = lora_splits(tiles * rt, a.K, sms, NW), chunks = a.K / 32;
    for (int item = blockIdx.x; item < tiles * rt * splits; item += gridDim.x) {
        const int split = item % splits, rest = item / splits, r0 = rest % rt * RR;
        const int4 tile = tile_of(plan, rest / rt, early);
        __syncthreads();  // (the previous item's sums and rows have been read)
        sm_order[tid] = early_row;
        const int* const row = tile.y + tile.z <= NW * 32 ? sm_order + tile.y : sm_row;
        if (row == sm_row && tid < tile.z) sm_row[tid] = __ldcg(order + tile.y + tid);
        const int rank = rank_of(a, tile.x);
        __syncthreads();
        const uint8_t* w = (const uint8_t*)a.a + ((int64_t)tile.x * a.rank + r0) * a.K * es;
        const int c0 = (int)((int64_t)chunks * split / splits), c1 = (int)((int64_t)chunks * (split + 1) / splits);
        const uint32_t ring = smem_u32(sm_sum) + warp * RING;
        // (few rows as 32: 40 rows of 12 fp32 adapters 24.7 us in place of 17.7, one row 6.0 in place of 4.8)
        if (tile.z <= 8)
            shrink_tile<F16, MT, 1>(a, row, tile.z, w, rank - r0, c0, c1, ring, sm_sum, PAD);
        else
            shrink_tile<F16, MT, 4>(a, row, tile.z, w, rank - r0, c0, c1, ring, sm_sum, PAD);
        __syncthreads();
        for (int i = tid; i < RR * tile.z; i += NW * 32) {
            const int r = i % RR, x = i / RR;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < NW; w++) sum += sm_sum[(w * RR + r) * PAD + x];
            if (r0 + r < a.rank) a.ws[((int64_t)split * rows + tile.y + x) * a.rank + r0 + r] = sum;
        }
    }
}

// ---------------------------------------------------------------- expand

// 2 V values of a row of B from shared memory in pairs (of fp32 weights as scaled parts, of the 8 V of four lanes; the root of the
// power that takes sums back).  left: how many the adapter's rank has from this lane's first on.
template <bool F16, int V>
__device__ __forceinline__ float weights(uint32_t at, int left, uint32_t (&hi)[V], uint32_t (&lo)[V]) {
    constexpr int W = F16 ? V : 2 * V;  // words
    uint32_t w[W];
    if constexpr (W >= 4) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 x = shared16(at + 4 * i);
            w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
        }
    } else if constexpr (W == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    } else {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
    }
    if constexpr (F16) {
#pragma unroll
        for (int i = 0; i < V; i++) hi[i] = w[i];
        if (__any_sync(0xffffffffu, left < 2 * V)) {
#pragma unroll
            for (int i = 0; i < V; i++) hi[i] &= (2 * i < left ? 0xFFFFu : 0u) | (2 * i + 1 < left ? 0xFFFF0000u : 0u);
        }
        return 1.f;
    } else {
        float x[2 * V], m = kLeast, down, up;
#pragma unroll
        for (int i = 0; i < 2 * V; i++) x[i] = i < left ? __uint_as_float(w[i]) : 0.f, m = fmaxf(m, fabsf(x[i]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        power_root(m, down, up);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float2 y = mul2(make_float2(x[2 * i], x[2 * i + 1]), both(down));
            split_h2(y.x, y.y, hi[i], lo[i]);
        }
        return up;
    }
}

// V: units of 8 ranks whose values a lane takes at once.  VEC: columns and rows allow 16-byte pieces.  NST: runs of 128 columns
// (16 of a warp) whose base and weights are on their way, in the warp's ring: a lane's own pieces of base, then the 16
// columns' rows of B as they lie in memory.
// A CTA takes an equal share of all (tile, run of columns), of one tile after another.
template <bool F16, int V, bool VEC, int NST, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) lora_expand_kernel(LoraArgs a, int max_tiles, int sms, int rr) {
    extern __shared__ __align__(16) uint4 sm_h[];  // [steps][2 row tiles][hi, lo][32 lanes], then the rings
    __shared__ int sm_row[kLoraTile];
    __shared__ float sm_up[kLoraTile];  // the powers of two that take the rows of h back (fp32 weights: their roots)
    constexpr int SG = (V + 1) / 2;     // matrix steps of a group of 8 V ranks
    constexpr int HR = kLoraTile / kWarps, HQ = kLoraMaxRank / 32;
    constexpr int es = F16 ? 2 : 4;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, j = lane >> 2;
    const int row_bytes = a.rank * es, stage = (VEC ? 2048 : 0) + 16 * row_bytes, steps = (a.rank + 8 * V - 1) / (8 * V) * SG;
    const uint32_t ring = smem_u32(sm_h) + steps * 2 * 64 * 16 + warp * NST * stage;
    const int* plan = (const int*)a.plan;
    const int4 head = __ldcg(reinterpret_cast<const int4*>(plan));
    const int4 early = first_tiles(plan, lane, max_tiles);
    const bool fits = head.w == lora_plan_sizes(a.n, a.adapters);
    const int tiles = !fits ? 0 : a.base && a.base == a.y ? head.y : head.x;  // in place, rows without an adapter stay as they are
    const int rows = head.z, splits = lora_splits(head.y * ((a.rank + rr - 1) / rr), a.K, sms, rr == 16 ? kShrinkWarps<F16, 1> : kShrinkWarps<F16, 2>), cols = (a.N + kCols - 1) / kCols;
    // The CTA's share: an equal one of all runs, the first CTAs one more, since they start first.  (Shares of one tile each save a
    // second preparation but not the time: 64 rows of 40 adapters took 0.5 us more, 40 rows of 12 0.7, 512 rows of one adapter 1.5
    // less.)
    const int64_t items = (int64_t)tiles * cols;
    const int ctas = gridDim.x, me = blockIdx.x;
    const int64_t each = items <= INT32_MAX ? (int64_t)((unsigned)items / (unsigned)ctas) : items / ctas, rest = items - each * ctas;
    int64_t item = each * me + min((int64_t)me, rest);
    const int64_t last = each * (me + 1) + min((int64_t)me + 1, rest);
    // this lane's first piece of 16 columns' weights: its column and byte within the row; and how far 512 bytes on is
    const int col0 = lane * 16 / row_bytes, byte0 = lane * 16 - col0 * row_bytes, col_step = 512 / row_bytes, byte_step = 512 - col_step * row_bytes;
    while (item < last) {
        const int which = items <= INT32_MAX ? (int)((unsigned)item / (unsigned)cols) : (int)(item / cols);
        const int run0 = (int)(item - (int64_t)which * cols), run1 = (int)min((int64_t)cols, run0 + (last - item));
        item += run1 - run0;
        const int4 tile = tile_of(plan, which, early);
        // what shrink does not write comes before the wait: the tile's rows, rank and scale, the first weights and the base's rows
        int my_row = 0;
        if (tid < tile.z) my_row = __ldcg(plan + plan_order(max_tiles) + tile.y + tid);
        const int rank = tile.x < 0 ? 0 : rank_of(a, tile.x);
        const float scale = tile.x >= 0 && a.scale ? __ldcg(a.scale + tile.x) : 1.f;
        const int mt = tile.z > 16 ? 2 : 1;
        const bool few = tile.z <= 8;
        const int groups = (rank + 8 * V - 1) / (8 * V), rank_bytes = rank * es;
        const uint8_t* const tile_b = (const uint8_t*)a.b + ((int64_t)tile.x * a.N + 16 * warp) * row_bytes;
        const unsigned run_bytes = kCols * row_bytes;
        auto fetch_b = [&](int run, int slot) {
            const uint32_t dst = ring + slot * stage + (VEC ? 2048 : 0);
            const int n0 = run * kCols + 16 * warp;
            const uint8_t* src = tile_b + (uint64_t)(unsigned)run * run_bytes;
#pragma unroll 1
            for (int x = lane * 16, col = col0, byte = byte0; x < 16 * row_bytes; x += 512) {
                const bool in = n0 + col < a.N && byte < rank_bytes;
                copy16(dst + x, in ? src + x : (const uint8_t*)a.b, in ? 16 : 0);
                col += col_step, byte += byte_step;
                if (byte >= row_bytes) col++, byte -= row_bytes;
            }
        };
        __syncthreads();  // (the previous tile's rows and operands have been read)
        if (tid < tile.z) sm_row[tid] = my_row;
        if (rank)
#pragma unroll 1
            for (int i = 0; i < NST; i++)
                if (run0 + i < run1) fetch_b(run0 + i, i);
        __syncthreads();
        int64_t at[4];  // rows j + 8 i
#pragma unroll
        for (int i = 0; i < 4; i++) at[i] = 8 * i + j < tile.z ? sm_row[8 * i + j] : -1;
        auto fetch_base = [&](int run, int slot) {
            const uint32_t dst = ring + slot * stage;
            const int n = run * kCols + 16 * warp + 4 * c;
            if (VEC && a.base)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (8 * i >= tile.z) break;
                    if (at[i] >= 0 && n < a.N) copy16(dst + i * 512 + lane * 16, a.base + at[i] * a.ldb + n, 16);
                }
        };
#pragma unroll 1
        for (int i = 0; i < NST; i++) {
            if (run0 + i < run1) fetch_base(run0 + i, i);
            copy_commit();
        }
        // h: a warp takes every eighth row, a lane every 32nd rank
        pdl_wait();
        float h[HR][HQ];
#pragma unroll
        for (int i = 0; i < HR; i++)
#pragma unroll
            for (int q = 0; q < HQ; q++) h[i][q] = 0.f;
        if (tile.x >= 0 && warp < tile.z) {
            const float* p = a.ws + ((int64_t)tile.y + warp) * a.rank + lane;
            const int64_t stride = (int64_t)rows * a.rank;
            // ranges on their way: eight of a row, two or four of four rows
            auto take = [&](auto in_flight, auto row_groups, auto rank_groups) {
                constexpr int S = decltype(in_flight)::value, R = decltype(row_groups)::value, Q = decltype(rank_groups)::value;
#pragma unroll 1
                for (int s0 = 0; s0 < splits; s0 += S, p += S * stride) {
                    float v[S][R][Q];
#pragma unroll
                    for (int s = 0; s < S; s++)
#pragma unroll
                        for (int i = 0; i < R; i++)
#pragma unroll
                            for (int q = 0; q < Q; q++) {
                                v[s][i][q] = 0.f;
                                if (s0 + s < splits && warp + kWarps * i < tile.z && lane + 32 * q < a.rank)
                                    v[s][i][q] = __ldcg(p + s * stride + (int64_t)kWarps * i * a.rank + 32 * q);
                            }
#pragma unroll
                    for (int s = 0; s < S; s++)
#pragma unroll
                        for (int i = 0; i < R; i++)
#pragma unroll
                            for (int q = 0; q < Q; q++) h[i][q] += v[s][i][q];
                }
            };
            const auto i1 = std::integral_constant<int, 1>{};
            if (few && a.rank <= 32)
                take(std::integral_constant<int, 8>{}, i1, i1);
            else if (few)
                take(std::integral_constant<int, 8>{}, i1, std::integral_constant<int, HQ>{});
            else if (a.rank <= 32)
                take(std::integral_constant<int, 4>{}, std::integral_constant<int, HR>{}, i1);
            else
                take(std::integral_constant<int, 2>{}, std::integral_constant<int, HR>{}, std::integral_constant<int, HQ>{});
        }
        // h as operands: value i of lane cc's 2 V in group g is rank 8 V g + 2 V cc + i, its pairs those of steps 0, 0, 1, 1
        const int held = groups * 8 * V;
#pragma unroll
        for (int x = 0; x < HR; x++) {
            const int row = warp + kWarps * x;
            if (row >= 16 * mt) break;
            float m = F16 ? 0.f : kLeast, down, up;
#pragma unroll
            for (int q = 0; q < HQ; q++) {
                h[x][q] = lane + 32 * q < rank ? h[x][q] * scale : 0.f;
                m = fmaxf(m, fabsf(h[x][q]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (F16)
                powers(m, down, up);
            else
                power_root(m, down, up);
            if (lane == 0) sm_up[row] = up;
#pragma unroll
            for (int q = 0; q < HQ; q++) {
                const int r = lane + 32 * q;
                if (32 * q >= held) break;
                uint32_t hi, lo;
                split_h2(h[x][q] * down, 0.f, hi, lo);
                const int g = r / (8 * V), cc = r % (8 * V) / (2 * V), i = r % (2 * V);
                unsigned short* dst = reinterpret_cast<unsigned short*>(sm_h + ((g * SG + i / 4) * 2 + row / 16) * 64 + (row & 7) * 4 + cc) +
                                      2 * (2 * (i / 2 & 1) + (row >> 3 & 1)) + (i & 1);
                if (r < held) {
                    dst[0] = (unsigned short)hi;
                    dst[32 * 8] = (unsigned short)lo;
                    if (V == 1) dst[4] = dst[32 * 8 + 4] = 0;  // (the step's other pairs)
                }
            }
        }
        __syncthreads();
        float up[4];
#pragma unroll
        for (int i = 0; i < 4; i++) up[i] = sm_up[min(8 * i, 16 * mt - 8) + j];
        int slot = 0;
#pragma unroll 1
        for (int run = run0; run < run1; run++) {
            copy_wait<NST - 1>();
            __syncwarp();  // the other lanes' pieces of B have landed
            const uint32_t st = ring + slot * stage;
            // column j of tile t is n0 + 4 (j / 2) + 2 t + j % 2, so that a lane's columns of both tiles are four neighbours
            const uint32_t wb = st + (VEC ? 2048 : 0) + (4 * (j >> 1) + (j & 1)) * row_bytes + 2 * V * c * es;
            float acc[2][2][4] = {};
#pragma unroll 1
            for (int g = 0; g < groups; g++) {
                uint32_t hi[2][V], lo[2][V];
                float2 back[2];  // of the lane's columns
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    const float u = weights<F16, V>(wb + 2 * t * row_bytes + g * 8 * V * es, rank - (8 * V * g + 2 * V * c), hi[t], lo[t]);
                    if (!F16) back[t] = make_float2(__shfl_sync(0xffffffffu, u, 8 * c), __shfl_sync(0xffffffffu, u, 8 * c + 4));
                }
                float sum[2][2][4] = {};
#pragma unroll
                for (int part = 1; part >= 0; part--)
#pragma unroll
                    for (int e = 0; e < SG; e++)
#pragma unroll
                        for (int m = 0; m < 2; m++) {
                            if (m >= mt) break;
                            const uint4 h = sm_h[((g * SG + e) * 2 + m) * 64 + part * 32 + lane];
#pragma unroll
                            for (int t = 0; t < 2; t++) {
                                const int x = 2 * e, y = V == 1 ? 0 : 2 * e + 1;  // (V = 1: h's second pairs are zeros)
                                if constexpr (!F16)
                                    if (part == 0) dot16(sum[m][t], h, lo[t][x], lo[t][y]);
                                dot16(sum[m][t], h, hi[t][x], hi[t][y]);
                            }
                        }
#pragma unroll
                for (int m = 0; m < 2; m++)
#pragma unroll
                    for (int t = 0; t < 2; t++)
                        if constexpr (F16) {
                            add4(acc[m][t], sum[m][t]);
                        } else {
#pragma unroll
                            for (int h = 0; h < 4; h += 2) {
                                const float2 z = back_from(make_float2(sum[m][t][h], sum[m][t][h + 1]), mul2(back[t], both(up[2 * m + h / 2])),
                                                           make_float2(acc[m][t][h], acc[m][t][h + 1]));
                                acc[m][t][h] = z.x, acc[m][t][h + 1] = z.y;
                            }
                        }
            }
            const int n = run * kCols + 16 * warp + 4 * c;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (8 * i >= tile.z) break;
                if (at[i] < 0 || n >= a.N) continue;
                const int m = i / 2, h = 2 * (i & 1);
                float4 v = make_float4(acc[m][0][h], acc[m][0][h + 1], acc[m][1][h], acc[m][1][h + 1]);
                if (F16) v.x *= up[i], v.y *= up[i], v.z *= up[i], v.w *= up[i];
                float* p = a.y + at[i] * a.ldy + n;
                if (VEC) {
                    if (a.base) {
                        const uint4 z = shared16(st + i * 512 + lane * 16);
                        v.x += __uint_as_float(z.x), v.y += __uint_as_float(z.y), v.z += __uint_as_float(z.z), v.w += __uint_as_float(z.w);
                    }
                    *reinterpret_cast<float4*>(p) = v;
                } else {
                    const float x[4] = {v.x, v.y, v.z, v.w}, *q = a.base + at[i] * a.ldb + n;
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if (n + k < a.N) p[k] = a.base ? __ldcg(q + k) + x[k] : x[k];
                }
            }
            __syncwarp();
            if (run + NST < run1) {
                if (rank) fetch_b(run + NST, slot);
                fetch_base(run + NST, slot);
            }
            copy_commit();
            slot = slot + 1 == NST ? 0 : slot + 1;
        }
    }
    pdl_wait();  // (also where there was nothing to do)
    if (!fits) {  // what the plan names may not be rows and adapters of this call: NaN, and no address is formed from it
        for (int64_t i = (int64_t)me * kThreads + tid; i < (int64_t)a.n * a.N; i += (int64_t)ctas * kThreads)
            a.y[i / a.N * a.ldy + i % a.N] = __int_as_float(0x7FC00000);
    }
    __threadfence();  // (and no early launch of the next kernel: y may be a cache, see launch_chained)
}

// Ranks of an item of shrink.  (2048 rows of fp32 adapters of rank 64 100 us, in items of 16 132: x is read once an item; one row of
// rank 16 4.8 us, in items of 32 5.9.)
int shrink_ranks(int rank) { return rank <= 16 ? 16 : 32; }

template <bool F16, int MT>
cudaError_t shrink(const LoraArgs& a, int max_tiles, cudaStream_t s) {
    constexpr int NW = kShrinkWarps<F16, MT>, RING = kRing<F16, MT>;
    auto k = lora_shrink_kernel<F16, MT>;
    static SmemOptIn opt;
    if (cudaError_t e = opt((const void*)k, NW * RING)) return e;
    return launch_chained(k, dim3(num_sms()), NW * 32, NW * RING, s, a, max_tiles, num_sms());
}

template <bool F16, int V, bool VEC, int NST, int CTAS>
cudaError_t expand_go(const LoraArgs& a, int max_tiles, int smem, cudaStream_t s) {
    auto k = lora_expand_kernel<F16, V, VEC, NST, CTAS>;
    static SmemOptIn opt;
    if (cudaError_t e = opt((const void*)k, CTAS == 2 ? kHalf : 220 * 1024)) return e;
    return launch_chained(k, dim3(CTAS * num_sms()), kThreads, smem, s, a, max_tiles, num_sms(), shrink_ranks(a.rank));
}

// Two CTAs to an SM where their rings fit it, with three runs on their way if those fit, else with two (64 rows of 4 fp16
// adapters of rank 64 beside 4096 -> 28672: 17.1 us; one CTA with two runs 19.0; 2048 rows of 5 of rank 32 97 and 117.  Four runs
// where they fit are no faster; two everywhere give 92.6 for those 2048 rows, 38.0 in place of 37.5 for 512 of rank 128, and the
// same for the others).  Two of
// one CTA's fit for every rank (128 fp32: 176 KB).
template <bool F16, int V, bool VEC>
cudaError_t expand(const LoraArgs& a, int max_tiles, cudaStream_t s) {
    const int operands = (a.rank + 8 * V - 1) / (8 * V) * ((V + 1) / 2) * 2 * 64 * 16, stage = (VEC ? 2048 : 0) + 16 * a.rank * (F16 ? 2 : 4);
    const int two = operands + 2 * kWarps * stage, three = two + kWarps * stage;
    if (three <= kHalf) return expand_go<F16, V, VEC, 3, 2>(a, max_tiles, three, s);
    if (two <= kHalf) return expand_go<F16, V, VEC, 2, 2>(a, max_tiles, two, s);
    return expand_go<F16, V, VEC, 2, 1>(a, max_tiles, two, s);
}
template <bool F16, int V>
cudaError_t expand(const LoraArgs& a, int max_tiles, bool vec, cudaStream_t s) {
    return vec ? expand<F16, V, true>(a, max_tiles, s) : expand<F16, V, false>(a, max_tiles, s);
}

template <bool F16>
cudaError_t lora(const LoraArgs& a, cudaStream_t s) {
    const int tiles = lora_max_tiles(a.n, a.adapters), rr = shrink_ranks(a.rank);
    cudaError_t e = rr == 16 ? shrink<F16, 1>(a, tiles, s) : shrink<F16, 2>(a, tiles, s);
    if (e) return e;
    const bool vec = a.N % 4 == 0 && a.ldy % 4 == 0 && (uintptr_t)a.y % 16 == 0 && (!a.base || (a.ldb % 4 == 0 && (uintptr_t)a.base % 16 == 0));
    // as many ranks a step as divide the rank (rank 64 by 8: 40 rows of 12 fp32 adapters 21.7 us in place of 17.7)
    if (a.rank % 32 == 0) return expand<F16, 4>(a, tiles, vec, s);
    if (a.rank % 16 == 0) return expand<F16, 2>(a, tiles, vec, s);
    return expand<F16, 1>(a, tiles, vec, s);
}

}  // namespace

size_t lora_plan_bytes(int n, int adapters) { return (plan_order(lora_max_tiles(n, adapters)) + n) * sizeof(int); }

cudaError_t launch_lora_plan(const int* ids, int n, int adapters, void* plan, cudaStream_t s) {
    return launch_chained(lora_plan_kernel, dim3(1), kPlanThreads, 0, s, ids, n, adapters, lora_max_tiles(n, adapters), (int*)plan);
}

// A range's sums of every row.  With t tiles there are at most SMs / t ranges, or one, and at most 32 t rows.
size_t lora_ws_bytes(int n, int rank) {
    return (size_t)std::min<int64_t>((int64_t)kMaxSplit * n, (int64_t)num_sms() * kLoraTile + n) * rank * sizeof(float);
}

cudaError_t launch_lora(const LoraArgs& a, cudaStream_t s) { return a.f16 ? lora<true>(a, s) : lora<false>(a, s); }

}  // namespace af

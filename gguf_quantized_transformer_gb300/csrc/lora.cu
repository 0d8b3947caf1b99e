// Low-rank adapters of many requests beside a shared projection: row i of the batch with adapter a,
//   y_i = base_i + scale_a B_a (A_a x_i),   A_a [rank, K], B_a [N, rank].
//
// The rows are put in the order of their adapters once a step (lora_plan_kernel: a counting sort), in tiles of up to 32 rows
// of one adapter, so that an adapter's weights are read once for all of them.  Then two kernels:
//  - shrink: h = A x.  A CTA takes a tile and a range of K, its warps chunks of 32 of that range in turn; weights and x go
//    from memory straight into operands (lane c of 4 owns 8 values of a chunk, on both sides, so the order within it is
//    free).  The warps' sums join in shared memory, the ranges' sums by their reader, both in order.
//  - expand: y = base + B (scale h).  A CTA takes a tile and runs of 128 columns; h's parts lie in shared memory as operands,
//    a warp's 16 columns of B come straight into operands, and y is moved in 16-byte pieces.
// Bound by the bytes of base, y and x for many rows, by those of the weights for few, and by two launches for one.
// Precision: tf32 products of parts.  fp16 weights are tf32 numbers; x, h and fp32 weights are cut into two parts of 11 bits
// (x = hi + lo to 2^-22), and the product of two lo parts is left out.  Tensor cores cut their sums: those of a chunk start
// from zero, small products first, and are added in fp32.
#include <algorithm>

#include "mma_sync.cuh"
#include "serve.cuh"
#include "tma.cuh"

namespace af {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxSplit = 16;
constexpr int kCols = 16 * kWarps;  // columns that a CTA of expand takes at once

__host__ __device__ inline int64_t plan_order(int max_tiles) { return 4 * (int64_t)(1 + max_tiles); }  // in ints

// ---------------------------------------------------------------- plan

__device__ __forceinline__ int cta_scan(int x, int& total) {  // inclusive
    __shared__ int part[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; w++) {
        if (w < warp) before += part[w];
        sum += part[w];
    }
    total = sum;
    return x + before;
}

__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(const int* __restrict__ ids, int n, int adapters, int max_tiles,
                                                                  int* __restrict__ plan) {
    __shared__ int count[kLoraMaxAdapters + 1], first[kLoraMaxAdapters + 2];  // rows of an adapter; its first tile
    const int t = threadIdx.x, lane = t & 31;
    pdl_launch_dependents();
    pdl_wait();
    for (int i = t; i <= adapters; i += kPlanThreads) count[i] = 0;
    __syncthreads();
    // rows of each adapter (those without one count as the last), a warp's equal ones at once
    auto bucket = [&](int i) {
        const int id = __ldcg(ids + i);
        return id >= 0 && id < adapters ? id : adapters;
    };
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + t, b = i < n ? bucket(i) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, b);
        if (b >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[b], __popc(same));
    }
    __syncthreads();
    int rows = 0, tiles = 0;
    const int bare = count[adapters];
    for (int i0 = 0; i0 <= adapters; i0 += kPlanThreads) {
        const int i = i0 + t, c = i <= adapters ? count[i] : 0;
        int total;
        const int r = cta_scan(c, total) + rows;
        rows += total;
        const int k = (c + kLoraTile - 1) / kLoraTile, f = cta_scan(k, total) + tiles;
        tiles += total;
        __syncthreads();
        if (i <= adapters) count[i] = r - c, first[i] = f - k;  // the adapter's first row and tile
    }
    if (t == 0) {
        first[adapters + 1] = tiles;
        const int bare_tiles = (bare + kLoraTile - 1) / kLoraTile;
        *reinterpret_cast<int4*>(plan) = make_int4(tiles, tiles - bare_tiles, n - bare, 0);
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
        const int i = i0 + t, b = i < n ? bucket(i) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, b);
        const int lead = __ffs(same) - 1;
        int at = 0;
        if (b >= 0 && lane == lead) at = atomicAdd(&count[b], __popc(same));
        at = __shfl_sync(0xffffffffu, at, lead);
        if (b >= 0) order[at + __popc(same & ((1u << lane) - 1))] = i;
    }
}

// ---------------------------------------------------------------- shrink

// Ranges of K: as many as two CTAs on every SM take at once, of at least 8 chunks of 32
__device__ __forceinline__ int lora_splits(int items, int K, int sms) {
    return max(1, min(min(2 * sms / max(items, 1), kMaxSplit), K / 32 / kWarps));
}

__device__ __forceinline__ int rank_of(const LoraArgs& a, int adapter) {
    return a.ranks ? min(max(__ldcg(a.ranks + adapter), 0), a.rank) : a.rank;
}
__device__ __forceinline__ float4 ldcg4(const float* p) { return __ldcg(reinterpret_cast<const float4*>(p)); }

// 8 weights of a row as tf32 parts; lo only of fp32 weights
template <bool F16>
struct Weights8 {
    uint4 w[F16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* p, bool in) {
#pragma unroll
        for (int i = 0; i < (F16 ? 1 : 2); i++)
            w[i] = in ? __ldcg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void parts(uint32_t (&hi)[8], uint32_t (&lo)[8]) const {
        if constexpr (F16) {
            const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
                hi[2 * i] = __float_as_uint(f.x), hi[2 * i + 1] = __float_as_uint(f.y);
            }
        } else {
            const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 8; i++) cut_tf32(__uint_as_float(x[i]), hi[i], lo[i]);
        }
    }
};

// The sums of chunks k0, k0 + kWarps .. below k1 for 16 MT ranks and 8 NT rows, U chunks on their way at once.
// wp: this lane's weights of rank j; in: the ranks that there are, from j on; xp: this lane's values of the rows 8 t + j, null
// where there is none.
template <bool F16, int MT, int NT, int U>
__device__ __forceinline__ void shrink_chunks(const uint8_t* wp, int in, int K, const float* const (&xp)[NT], int k0, int k1,
                                              float (&acc)[MT][NT][4]) {
    constexpr size_t es = F16 ? 2 : 4;
#pragma unroll 1
    for (int k = k0; k < k1; k += U * kWarps) {
        Weights8<F16> w[U][MT][2];
        float4 x[U][NT][2];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int ku = k + u * kWarps;
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    w[u][m][h].load(wp + ((int64_t)(16 * m + 8 * h) * K + 32 * ku) * es, ku < k1 && 16 * m + 8 * h < in);
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int i = 0; i < 2; i++)
                    x[u][t][i] = ku < k1 && xp[t] ? ldcg4(xp[t] + 32 * ku + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (u && k + u * kWarps >= k1) break;
#pragma unroll
            for (int m = 0; m < MT; m++) {
                uint32_t h0[8], l0[8], h1[8], l1[8];
                w[u][m][0].parts(h0, l0);
                w[u][m][1].parts(h1, l1);
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    const float4 a = x[u][t][0], b = x[u][t][1];
                    const float xs[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                    uint32_t xh[8], xl[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) cut_tf32(xs[i], xh[i], xl[i]);
                    float sum[4];
                    mma8z(sum, make_uint4(h0[0], h1[0], h0[1], h1[1]), xl[0], xl[1]);
#pragma unroll
                    for (int e = 2; e < 8; e += 2) mma8(sum, make_uint4(h0[e], h1[e], h0[e + 1], h1[e + 1]), xl[e], xl[e + 1]);
                    if constexpr (!F16) {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) mma8(sum, make_uint4(l0[e], l1[e], l0[e + 1], l1[e + 1]), xh[e], xh[e + 1]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; e += 2) mma8(sum, make_uint4(h0[e], h1[e], h0[e + 1], h1[e + 1]), xh[e], xh[e + 1]);
                    add4(acc[m][t], sum);
                }
            }
        }
    }
}

// The tile's rows' 16 MT ranks, summed over the warps, in `sum`: [warps][16 MT][PAD]
template <bool F16, int MT, int NT, int U>
__device__ __forceinline__ void shrink_tile(const LoraArgs& a, const int* row, int count, const uint8_t* wp, int in, int k0, int k1,
                                            float* sum, int pad) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, j = lane >> 2;
    const float* xp[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) xp[t] = 8 * t + j < count ? a.x + (int64_t)row[8 * t + j] * a.ldx + 8 * c : nullptr;
    float acc[MT][NT][4] = {};
    shrink_chunks<F16, MT, NT, U>(wp, in, a.K, xp, k0 + warp, k1, acc);
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
__global__ void __launch_bounds__(kThreads, 2) lora_shrink_kernel(LoraArgs a, int max_tiles, int sms) {
    constexpr int RR = 16 * MT, PAD = kLoraTile + 2;
    extern __shared__ __align__(16) float sm_sum[];  // [warps][RR][PAD]
    __shared__ int sm_row[kLoraTile];
    const int tid = threadIdx.x, lane = tid & 31, c = lane & 3, j = lane >> 2;
    const int* plan = (const int*)a.plan;
    pdl_launch_dependents();
    pdl_wait();
    const int4 head = __ldcg(reinterpret_cast<const int4*>(plan));
    const int tiles = head.y, rows = head.z, rt = (a.rank + RR - 1) / RR;
    const int splits = lora_splits(tiles * rt, a.K, sms), chunks = a.K / 32;
    const size_t es = F16 ? 2 : 4;
    for (int item = blockIdx.x; item < tiles * rt * splits; item += gridDim.x) {
        const int split = item % splits, rest = item / splits, r0 = rest % rt * RR;
        const int4 tile = __ldcg(reinterpret_cast<const int4*>(plan) + 1 + rest / rt);
        __syncthreads();  // (the previous item's sums and rows have been read)
        if (tid < tile.z) sm_row[tid] = __ldcg(plan + plan_order(max_tiles) + tile.y + tid);
        const int rank = rank_of(a, tile.x);
        __syncthreads();
        const uint8_t* wp = (const uint8_t*)a.a + ((int64_t)tile.x * a.rank + r0 + j) * a.K * es + 8 * c * es;
        const int c0 = (int)((int64_t)chunks * split / splits), c1 = (int)((int64_t)chunks * (split + 1) / splits);
        if (tile.z <= 8)
            shrink_tile<F16, MT, 1, F16 && MT == 1 ? 4 : 2>(a, sm_row, tile.z, wp, rank - r0 - j, c0, c1, sm_sum, PAD);
        else
            shrink_tile<F16, MT, 4, 1>(a, sm_row, tile.z, wp, rank - r0 - j, c0, c1, sm_sum, PAD);
        __syncthreads();
        for (int i = tid; i < RR * tile.z; i += kThreads) {
            const int r = i % RR, row = i / RR;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; w++) sum += sm_sum[(w * RR + r) * PAD + row];
            if (r0 + r < a.rank) a.ws[((int64_t)split * rows + tile.y + row) * a.rank + r0 + r] = sum;
        }
    }
}

// ---------------------------------------------------------------- expand

// 2 V values of a row of B from p on, as tf32 parts.  left: how many of them the adapter's rank has.
template <bool F16, int V>
struct WeightsV {
    static constexpr int W = F16 ? V : 2 * V;  // words
    uint32_t w[W];
    __device__ __forceinline__ void load(const void* p, bool in) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
        if constexpr (W >= 4) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 x = in ? __ldcg(reinterpret_cast<const uint4*>(q + i)) : make_uint4(0u, 0u, 0u, 0u);
                w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
            }
        } else if constexpr (W == 2) {
            const uint2 x = in ? __ldcg(reinterpret_cast<const uint2*>(q)) : make_uint2(0u, 0u);
            w[0] = x.x, w[1] = x.y;
        } else {
            w[0] = in ? __ldcg(q) : 0u;
        }
    }
    __device__ __forceinline__ void parts(uint32_t (&hi)[2 * V], uint32_t (&lo)[2 * V], int left) const {
#pragma unroll
        for (int i = 0; i < 2 * V; i++) {
            float f;
            if constexpr (F16)
                f = __half2float(__ushort_as_half((unsigned short)(w[i / 2] >> (16 * (i & 1)))));
            else
                f = __uint_as_float(w[i]);
            if (i >= left) f = 0.f;
            if (F16)
                hi[i] = __float_as_uint(f);
            else
                cut_tf32(f, hi[i], lo[i]);
        }
    }
};

// V: units of 8 ranks whose values a lane loads at once.  VEC: columns and rows allow 16-byte pieces.
// Block (x, y) takes runs of kCols columns of tile y: `runs` of them from x runs on.  The next run's base and the next weights
// are on their way while this run's products are formed.
template <bool F16, int V, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) lora_expand_kernel(LoraArgs a, int max_tiles, int sms, int rr, int runs) {
    extern __shared__ __align__(16) uint4 sm_h[];  // [steps][2 row tiles][hi, lo][32 lanes]
    __shared__ int sm_row[kLoraTile];
    constexpr size_t es = F16 ? 2 : 4;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, j = lane >> 2;
    const int* plan = (const int*)a.plan;
    pdl_launch_dependents();
    pdl_wait();
    const int4 head = __ldcg(reinterpret_cast<const int4*>(plan)), tile = __ldcg(reinterpret_cast<const int4*>(plan) + 1 + blockIdx.y);
    if ((int)blockIdx.y >= head.x || (tile.x < 0 && a.base == a.y)) return;  // (in place, rows without an adapter stay)
    const int rank = tile.x < 0 ? 0 : rank_of(a, tile.x);
    const int groups = (rank + 8 * V - 1) / (8 * V), mt = tile.z > 16 ? 2 : 1;
    const int end = min(a.N, (int)(blockIdx.x + 1) * runs * kCols);
    int n0 = blockIdx.x * runs * kCols + 16 * warp;
    // column j of tile t is n0 + 4 (j / 2) + 2 t + j % 2, so that a lane's columns of both tiles are four neighbours
    WeightsV<F16, V> w[2];
    auto load_w = [&](int n, int g) {
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const int col = n + 4 * (j >> 1) + 2 * t + (j & 1);
            const bool in = g < groups && col < end;
            w[t].load((const uint8_t*)a.b + (((int64_t)tile.x * a.N + (in ? col : 0)) * a.rank + 8 * V * g + 2 * V * c) * es, in);
        }
    };
    if (groups) load_w(n0, 0);
    if (tid < tile.z) sm_row[tid] = __ldcg(plan + plan_order(max_tiles) + tile.y + tid);
    // h as operands: value i of lane cc's 2 V in group g is rank 8 V g + 2 V cc + i
    if (groups) {
        const float scale = a.scale ? __ldcg(a.scale + tile.x) : 1.f;
        const int rows = head.z, splits = lora_splits(head.y * ((a.rank + rr - 1) / rr), a.K, sms), held = groups * 8 * V;
        const int64_t stride = (int64_t)rows * a.rank;
        for (int i = tid; i < held * 16 * mt; i += kThreads) {
            const int row = i / held, r = i - row * held;
            float h = 0.f;
            if (r < rank && row < tile.z) {
                const float* p = a.ws + ((int64_t)tile.y + row) * a.rank + r;
#pragma unroll 4
                for (int s = 0; s < splits; s++) h += __ldcg(p + s * stride);
                h *= scale;
            }
            uint32_t hi, lo;
            cut_tf32(h, hi, lo);
            const int g = r / (8 * V), cc = r % (8 * V) / (2 * V), k = r % (2 * V);
            uint32_t* dst = reinterpret_cast<uint32_t*>(sm_h + ((g * V + k / 2) * 2 + row / 16) * 64 + (row & 7) * 4 + cc) +
                            (row >> 3 & 1) + 2 * (k & 1);
            dst[0] = hi;
            dst[32 * 4] = lo;
        }
    }
    __syncthreads();
    // base: rows j + 8 i, columns n0 + 4 c ..
    int64_t at[4];
#pragma unroll
    for (int i = 0; i < 4; i++) at[i] = 8 * i + j < tile.z ? sm_row[8 * i + j] : -1;
    float4 y[4];
    auto load_base = [&](int n) {
        n += 4 * c;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!a.base || at[i] < 0 || n >= end) continue;
            const float* p = a.base + at[i] * a.ldb + n;
            if (VEC) {
                y[i] = ldcg4(p);
            } else {
                y[i].x = __ldcg(p);
                if (n + 1 < end) y[i].y = __ldcg(p + 1);
                if (n + 2 < end) y[i].z = __ldcg(p + 2);
                if (n + 3 < end) y[i].w = __ldcg(p + 3);
            }
        }
    };
    load_base(n0);
#pragma unroll 1
    for (; n0 < end; n0 += kCols) {
        float4 z[4];
#pragma unroll
        for (int i = 0; i < 4; i++) z[i] = y[i];
        if (n0 + kCols < end) load_base(n0 + kCols);
        float acc[2][2][4] = {};
#pragma unroll 1
        for (int g = 0; g < groups; g++) {
            uint32_t hi[2][2 * V], lo[2][2 * V];
#pragma unroll
            for (int t = 0; t < 2; t++) w[t].parts(hi[t], lo[t], rank - (8 * V * g + 2 * V * c));
            if (g + 1 < groups)
                load_w(n0, g + 1);
            else if (n0 + kCols < end)
                load_w(n0 + kCols, 0);
#pragma unroll
            for (int m = 0; m < 2; m++) {
                if (m >= mt) break;
                float sum[2][4] = {};
#pragma unroll
                for (int part = 1; part >= 0; part--)
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        const uint4 h = sm_h[((g * V + e) * 2 + m) * 64 + part * 32 + lane];
#pragma unroll
                        for (int t = 0; t < 2; t++) {
                            if (!F16 && part == 0) mma8(sum[t], h, lo[t][2 * e], lo[t][2 * e + 1]);
                            mma8(sum[t], h, hi[t][2 * e], hi[t][2 * e + 1]);
                        }
                    }
#pragma unroll
                for (int t = 0; t < 2; t++) add4(acc[m][t], sum[t]);
            }
        }
        const int n = n0 + 4 * c;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (at[i] < 0 || n >= end) continue;
            const int m = i / 2, h = 2 * (i & 1);
            float* p = a.y + at[i] * a.ldy + n;
            const float4 v = make_float4(z[i].x + acc[m][0][h], z[i].y + acc[m][0][h + 1], z[i].z + acc[m][1][h], z[i].w + acc[m][1][h + 1]);
            if (VEC) {
                *reinterpret_cast<float4*>(p) = v;
            } else {
                p[0] = v.x;
                if (n + 1 < end) p[1] = v.y;
                if (n + 2 < end) p[2] = v.z;
                if (n + 3 < end) p[3] = v.w;
            }
        }
    }
}

// ranks of a shrink item
int shrink_ranks(int rank) { return rank <= 16 ? 16 : 32; }

template <bool F16, int MT>
cudaError_t shrink(const LoraArgs& a, int max_tiles, cudaStream_t s) {
    constexpr int smem = kWarps * 16 * MT * (kLoraTile + 2) * 4;
    auto k = lora_shrink_kernel<F16, MT>;
    static SmemOptIn opt;
    if (cudaError_t e = opt((const void*)k, smem)) return e;
    return launch_chained(k, dim3(2 * num_sms()), kThreads, smem, s, a, max_tiles, num_sms());
}

template <bool F16, int V>
cudaError_t expand(const LoraArgs& a, int max_tiles, bool vec, cudaStream_t s) {
    const int smem = (a.rank + 8 * V - 1) / (8 * V) * V * 2 * 64 * 16;  // at most 32 KB
    // runs of columns for a CTA: four where that leaves two CTAs for every SM
    const int64_t cols = (a.N + kCols - 1) / kCols;
    const int runs = (cols + 3) / 4 * ((a.n + kLoraTile - 1) / kLoraTile) >= 2 * num_sms() ? 4 : 1;
    const dim3 grid((unsigned)((cols + runs - 1) / runs), max_tiles);
    auto go = [&](auto k) { return launch_chained(k, grid, kThreads, smem, s, a, max_tiles, num_sms(), shrink_ranks(a.rank), runs); };
    return vec ? go(lora_expand_kernel<F16, V, true>) : go(lora_expand_kernel<F16, V, false>);
}

template <bool F16>
cudaError_t lora(const LoraArgs& a, cudaStream_t s) {
    const int tiles = lora_max_tiles(a.n, a.adapters), rr = shrink_ranks(a.rank);
    cudaError_t e = rr == 16 ? shrink<F16, 1>(a, tiles, s) : shrink<F16, 2>(a, tiles, s);
    if (e) return e;
    const bool vec = a.N % 4 == 0 && a.ldy % 4 == 0 && (uintptr_t)a.y % 16 == 0 && (!a.base || (a.ldb % 4 == 0 && (uintptr_t)a.base % 16 == 0));
    if (a.rank % 32 == 0) return expand<F16, 4>(a, tiles, vec, s);
    if (a.rank % 16 == 0) return expand<F16, 2>(a, tiles, vec, s);
    return expand<F16, 1>(a, tiles, vec, s);
}

}  // namespace

size_t lora_plan_bytes(int n, int adapters) { return (plan_order(lora_max_tiles(n, adapters)) + n) * sizeof(int); }

cudaError_t launch_lora_plan(const int* ids, int n, int adapters, void* plan, cudaStream_t s) {
    return launch_chained(lora_plan_kernel, dim3(1), kPlanThreads, 0, s, ids, n, adapters, lora_max_tiles(n, adapters), (int*)plan);
}

// A range's sums of every row.  With t tiles there are at most 2 SMs / t ranges, or one, and at most 32 t rows.
size_t lora_ws_bytes(int n, int rank) {
    return (size_t)std::min<int64_t>((int64_t)kMaxSplit * n, 2 * (int64_t)num_sms() * kLoraTile + n) * rank * sizeof(float);
}

cudaError_t launch_lora(const LoraArgs& a, cudaStream_t s) { return a.f16 ? lora<true>(a, s) : lora<false>(a, s); }

}  // namespace af

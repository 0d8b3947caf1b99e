// Low-rank adapters of many requests beside a shared projection: row i of the batch with adapter a,
//   y_i = base_i + scale_a B_a (A_a x_i),   A_a [rank, K], B_a [N, rank].
//
// The rows are put in the order of their adapters once a step (lora_plan_kernel: a counting sort), in tiles of up to 32 rows
// of one adapter, so that an adapter's weights are read once for all of them.  Then two kernels:
//  - shrink: h = A x.  A CTA takes a tile and a range of K, its warps chunks of 32 of that range in turn; weights and x go
//    from memory straight into operands (lane c of 4 owns 8 values of a chunk, on both sides, so the order within it is
//    free).  The warps' sums join in shared memory, the ranges' sums by their reader, both in order.
//  - expand: y = base + B (scale h).  A CTA takes a run of (tile, 128 columns); h's parts lie in shared memory as operands,
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
constexpr int kCols = 16 * kWarps;  // columns of an expand item

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

// Ranges of K: as many as bring two CTAs to every SM, of at least 8 chunks of 32
__device__ __forceinline__ int lora_splits(int tiles, int K, int sms) {
    const int want = (2 * sms + tiles - 1) / max(tiles, 1);
    return max(1, min(min(want, kMaxSplit), K / 32 / kWarps));
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

template <bool F16, int MT>
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(LoraArgs a, int max_tiles, int sms) {
    constexpr int NT = kLoraTile / 8, RR = 16 * MT, PAD = kLoraTile + 2;
    extern __shared__ __align__(16) float sm_sum[];  // [warps][RR][PAD]
    __shared__ int sm_row[kLoraTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, j = lane >> 2;
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
        const int rank = rank_of(a, tile.x);
        __syncthreads();  // (the previous item's sums and rows have been read)
        if (tid < tile.z) sm_row[tid] = __ldcg(plan + plan_order(max_tiles) + tile.y + tid);
        __syncthreads();
        const int nt = (tile.z + 7) / 8;
        const float* xp[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) xp[t] = a.x + (8 * t + j < tile.z ? (int64_t)sm_row[8 * t + j] * a.ldx : 0) + 8 * c;
        const uint8_t* wp = (const uint8_t*)a.a + ((int64_t)tile.x * a.rank + r0 + j) * a.K * es + 8 * c * es;
        const int c0 = (int)((int64_t)chunks * split / splits), c1 = (int)((int64_t)chunks * (split + 1) / splits);
        float acc[MT][NT][4] = {};
        for (int k = c0 + warp; k < c1; k += kWarps) {
            Weights8<F16> w[MT][2];
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    w[m][h].load(wp + ((int64_t)(16 * m + 8 * h) * a.K + 32 * k) * es, r0 + 16 * m + 8 * h + j < rank);
            float4 x[NT][2];
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int i = 0; i < 2; i++)
                    x[t][i] = t < nt && 8 * t + j < tile.z ? ldcg4(xp[t] + 32 * k + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int m = 0; m < MT; m++) {
                uint32_t h0[8], l0[8], h1[8], l1[8];
                w[m][0].parts(h0, l0);
                w[m][1].parts(h1, l1);
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    if (t >= nt) break;
                    const float xs[8] = {x[t][0].x, x[t][0].y, x[t][0].z, x[t][0].w, x[t][1].x, x[t][1].y, x[t][1].z, x[t][1].w};
                    uint32_t xh[8], xl[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) cut_tf32(xs[i], xh[i], xl[i]);
                    float sum[4] = {};
#pragma unroll
                    for (int e = 0; e < 8; e += 2) mma8(sum, make_uint4(h0[e], h1[e], h0[e + 1], h1[e + 1]), xl[e], xl[e + 1]);
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
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    if (t < nt)
                        *reinterpret_cast<float2*>(sm_sum + (warp * RR + 16 * m + 8 * h + j) * PAD + 8 * t + 2 * c) =
                            make_float2(acc[m][t][2 * h], acc[m][t][2 * h + 1]);
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
template <bool F16, int V, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) lora_expand_kernel(LoraArgs a, int max_tiles, int sms, int rr) {
    extern __shared__ __align__(16) uint4 sm_h[];  // [steps][2 row tiles][hi, lo][32 lanes]
    __shared__ int sm_row[kLoraTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, j = lane >> 2;
    const int* plan = (const int*)a.plan;
    pdl_launch_dependents();
    pdl_wait();
    const int4 head = __ldcg(reinterpret_cast<const int4*>(plan));
    const int tiles = a.base == a.y && a.base ? head.y : head.x;  // in place, rows without an adapter stay as they are
    const int rows = head.z, splits = lora_splits(head.y * ((a.rank + rr - 1) / rr), a.K, sms);
    const int cols = (a.N + kCols - 1) / kCols;
    const int64_t items = (int64_t)tiles * cols;
    const size_t es = F16 ? 2 : 4;
    int have = -1;  // the tile in shared memory
    int4 tile = make_int4(-1, 0, 0, 0);
    int rank = 0;
    for (int64_t item = items * blockIdx.x / gridDim.x; item < items * (blockIdx.x + 1) / gridDim.x; item++) {
        const int at = (int)(item / cols), n0 = (int)(item % cols) * kCols + 16 * warp;
        if (at != have) {
            have = at;
            tile = __ldcg(reinterpret_cast<const int4*>(plan) + 1 + at);
            rank = tile.x < 0 ? 0 : rank_of(a, tile.x);
            const float scale = tile.x >= 0 && a.scale ? __ldcg(a.scale + tile.x) : 1.f;
            __syncthreads();
            if (tid < tile.z) sm_row[tid] = __ldcg(plan + plan_order(max_tiles) + tile.y + tid);
            // h as operands: value i of lane cc's 2 V in group g is rank 8 V g + 2 V cc + i
            const int groups = (rank + 8 * V - 1) / (8 * V);
            for (int i = tid; i < groups * 8 * V * kLoraTile; i += kThreads) {
                const int r = i % (groups * 8 * V), row = i / (groups * 8 * V);
                float h = 0.f;
                if (r < rank && row < tile.z) {
                    const float* p = a.ws + ((int64_t)tile.y + row) * a.rank + r;
                    for (int s = 0; s < splits; s++) h += __ldcg(p + (int64_t)s * rows * a.rank);
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
            __syncthreads();
        }
        if (n0 >= a.N) continue;
        const int groups = (rank + 8 * V - 1) / (8 * V), mt = tile.z > 16 ? 2 : 1;
        // base, on its way while the products run: rows j + 8 i, columns 4 c ..
        float4 y[4];
        const int n = n0 + 4 * c;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (a.base && 8 * i + j < tile.z) {
                const float* p = a.base + (int64_t)sm_row[8 * i + j] * a.ldb + n;
                if (VEC) {
                    if (n < a.N) y[i] = ldcg4(p);
                } else {
                    if (n < a.N) y[i].x = __ldcg(p);
                    if (n + 1 < a.N) y[i].y = __ldcg(p + 1);
                    if (n + 2 < a.N) y[i].z = __ldcg(p + 2);
                    if (n + 3 < a.N) y[i].w = __ldcg(p + 3);
                }
            }
        }
        float acc[2][2][4] = {};
        // column j of tile t is n0 + 4 (j / 2) + 2 t + j % 2, so that a lane's columns of both tiles are four neighbours
        const uint8_t* bp[2];
        bool in[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const int col = n0 + 4 * (j >> 1) + 2 * t + (j & 1);
            in[t] = col < a.N && tile.x >= 0;
            bp[t] = (const uint8_t*)a.b + (((int64_t)max(tile.x, 0) * a.N + (in[t] ? col : 0)) * a.rank + 2 * V * c) * es;
        }
        for (int g = 0; g < groups; g++) {
            WeightsV<F16, V> w[2];
#pragma unroll
            for (int t = 0; t < 2; t++) w[t].load(bp[t] + (size_t)g * 8 * V * es, in[t]);
            uint32_t hi[2][2 * V], lo[2][2 * V];
#pragma unroll
            for (int t = 0; t < 2; t++) w[t].parts(hi[t], lo[t], rank - (8 * V * g + 2 * V * c));
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
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (8 * i + j >= tile.z) continue;
            const int m = i / 2, h = 2 * (i & 1);
            float* p = a.y + (int64_t)sm_row[8 * i + j] * a.ldy + n;
            const float4 v = make_float4(y[i].x + acc[m][0][h], y[i].y + acc[m][0][h + 1], y[i].z + acc[m][1][h],
                                         y[i].w + acc[m][1][h + 1]);
            if (VEC) {
                if (n < a.N) *reinterpret_cast<float4*>(p) = v;
            } else {
                if (n < a.N) p[0] = v.x;
                if (n + 1 < a.N) p[1] = v.y;
                if (n + 2 < a.N) p[2] = v.z;
                if (n + 3 < a.N) p[3] = v.w;
            }
        }
    }
}

// ranks of a shrink item: 16, 32 or 64
int shrink_ranks(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : 64; }

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
    auto go = [&](auto k) { return launch_chained(k, dim3(2 * num_sms()), kThreads, smem, s, a, max_tiles, num_sms(), shrink_ranks(a.rank)); };
    return vec ? go(lora_expand_kernel<F16, V, true>) : go(lora_expand_kernel<F16, V, false>);
}

template <bool F16>
cudaError_t lora(const LoraArgs& a, cudaStream_t s) {
    const int tiles = lora_max_tiles(a.n, a.adapters), rr = shrink_ranks(a.rank);
    cudaError_t e = rr == 16 ? shrink<F16, 1>(a, tiles, s) : rr == 32 ? shrink<F16, 2>(a, tiles, s) : shrink<F16, 4>(a, tiles, s);
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

// A range's sums of every row.  With t tiles there are at most 2 SMs / t + 1 ranges, and at most 32 t rows.
size_t lora_ws_bytes(int n, int rank) {
    return (size_t)std::min<int64_t>((int64_t)kMaxSplit * n, 2 * (int64_t)num_sms() * kLoraTile + n) * rank * sizeof(float);
}

cudaError_t launch_lora(const LoraArgs& a, cudaStream_t s) { return a.f16 ? lora<true>(a, s) : lora<false>(a, s); }

}  // namespace af

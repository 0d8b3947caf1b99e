// The step of a serving loop that maps new tokens to slots of a paged cache: request i holds len_i tokens in the pages
// that its table row names, page_size to a page.  Its new tokens get the rows start_i .. of the batch; a token at position p
// lies in slot page * page_size + p % page_size.  Pages come from the head of a ring of free ones, in the requests' order,
// and those of ended requests go behind its last one, so that no entry that is read here is written here.
//
// Three prefix sums over the requests (rows, pages taken, pages given back), one CTA; then one
// thread per row of the batch, which finds its request by a binary search over the rows' starts.  A new page begins with a
// new token, so the thread of the page's first token writes the table.  Small steps do both in the one CTA, larger ones the
// second part in a grid of their own.
// Latency-bound: one or two launches, three rounds of dependent loads (lengths; requests; pages), the barriers of the sums.  In
// one CTA 64 requests take 3.0 us and a step of 256 in which 16 end and give back 4000 pages 6.2; 24 prompts with 414,896 rows, in
// two launches, 7.3, of which the 5 MB of slots, positions and requests are 0.7.  (In a graph of such calls; launched one by one 4.5,
// 6.3 and 7.7 to 10.)
#include <algorithm>

#include "serve.cuh"
#include "tma.cuh"

namespace af {

namespace {

// Threads of the scanning CTA: fewer where it does both parts for up to 512 requests.  (64 requests with a token
// each 3.0 us with 512, 3.4 with 1024, which issue twice the instructions; with 11 tokens each 4.0 and 3.5.  Before a second launch
// 512 are slower outside a graph: 124 requests 9.1 and 7.6 us, 2000 requests 12.6 and 11.5; in a graph 64 requests with 2656 rows
// take 5.8 and 6.2, 2000 requests 12.0 and 11.0.)
constexpr int kFewSeqs = 512, kScan = 1024;
constexpr int kFillRows = 4, kFill = 256;  // rows of a thread at a time, threads of a CTA of the second part
constexpr int kKept = 2048;                // requests whose prefix sums a CTA of the second part keeps

// A request as the second part sees it: .x the first page it takes (an index behind the ring's head), kRefused or kEnded;
// .y its tokens before the step, .z its pages before the step, .w pages given back by earlier requests
constexpr int kRefused = -1, kEnded = -2;

__device__ __forceinline__ int64_t clamp_int(int64_t x) { return x < INT32_MAX ? x : INT32_MAX; }

// Sum over the warp of values below 2^40
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
    return ((int64_t)__reduce_add_sync(0xffffffffu, (unsigned)(x >> 24)) << 24) + __reduce_add_sync(0xffffffffu, (unsigned)x & 0xFFFFFFu);
}

// Inclusive prefix sums over the CTA of three values a thread, each below 2^31; `total` receives the CTA's.  live: the warp's may be
// other than zeros.
template <int T>
__device__ __forceinline__ void cta_scan(bool live, int64_t (&x)[3], int64_t (&total)[3]) {
    __shared__ int64_t part[T / 32][3];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (live) {
#pragma unroll
        for (int o = 1; o < 32; o *= 2)
#pragma unroll
            for (int k = 0; k < 3; k++) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
                if (lane >= o) x[k] += y;
            }
    }
    __syncthreads();  // (the previous call's parts have been read)
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < 3; k++) part[warp][k] = x[k];
    __syncthreads();
    // every warp sums the others' parts, lane by lane
#pragma unroll
    for (int k = 0; k < 3; k++) {
        const int64_t y = lane < T / 32 ? part[lane][k] : 0;
        total[k] = warp_sum(y);
        if (live) x[k] += warp_sum(lane < warp ? y : 0);
    }
}

// For N numbers x: the last i of [0, n) with key(i) <= x; key(0) <= x
template <int N, typename F>
__device__ __forceinline__ void last_le(int n, const int (&x)[N], int (&i)[N], F key) {
#pragma unroll
    for (int k = 0; k < N; k++) i[k] = 0;
    for (int w = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; w; w >>= 1)
#pragma unroll
        for (int k = 0; k < N; k++)
            if (i[k] + w < n && key(i[k] + w) <= x[k]) i[k] += w;
}

__device__ __forceinline__ int page_of(const PagesArgs& a, int pos) {
    return a.page_mul ? (int)(__umulhi((unsigned)pos, a.page_mul) >> a.page_shift) : pos;
}
// Pages that hold x tokens
__device__ __forceinline__ int pages_for(const PagesArgs& a, int x) {
    const int e = page_of(a, x);
    return e + (e * a.page != x ? 1 : 0);
}

// x modulo n, for x < 2 n
__device__ __forceinline__ int wrap(unsigned x, int n) { return (int)(x >= (unsigned)n ? x - (unsigned)n : x); }

// Rows and returned pages of thread t of nt: ROWS neighbours at a time.  start(i), back(i): the prefix sums; head, count: the
// ring before the step.
template <int ROWS, typename S, typename B, typename Q>
__device__ __forceinline__ void fill(const PagesArgs& a, int64_t t, int64_t nt, int total, int returned, int head, int count, S start,
                                     B back, Q request) {
    for (int64_t at = t * ROWS; at < a.rows; at += nt * ROWS) {
        const int r0 = (int)at;
        int slot[ROWS], pos[ROWS], seq[ROWS];
        int i = 0, begin = 0, end = -1;  // rows [begin, end) of request i
        if (r0 < total) {
            const int x[1] = {r0};
            int y[1];
            last_le<1>(a.n, x, y, start);
            i = y[0];
        }
        int4 q = make_int4(kRefused, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < ROWS; k++) {
            const int r = r0 + k;
            slot[k] = pos[k] = seq[k] = -1;
            if (r >= total || at + k >= a.rows) continue;
            if (r >= end) {
                if (k) {
                    do i++;
                    while (i + 1 < a.n && start(i + 1) <= r);
                }
                begin = start(i);
                end = i + 1 < a.n ? start(i + 1) : total;
                q = request(i);
            }
            if (q.x < 0) continue;
            const int p = q.y + (r - begin), e = page_of(a, p);
            const int off = p - e * a.page;
            int page;
            if (e < q.z) {
                page = __ldcg(a.table + (int64_t)i * a.width + e);
            } else {
                page = __ldcg(a.free + wrap((unsigned)head + (unsigned)(q.x + (e - q.z)), a.n_pages));
                if (off == 0) a.table[(int64_t)i * a.width + e] = page;
            }
            slot[k] = page >= 0 && page < a.n_pages ? page * a.page + off : -1;
            pos[k] = p;
            seq[k] = i;
        }
        if (ROWS == 4 && at + ROWS <= a.rows && a.vec) {
            *reinterpret_cast<int4*>(a.slots + r0) = make_int4(slot[0], slot[1 % ROWS], slot[2 % ROWS], slot[3 % ROWS]);
            *reinterpret_cast<int4*>(a.pos + r0) = make_int4(pos[0], pos[1 % ROWS], pos[2 % ROWS], pos[3 % ROWS]);
            *reinterpret_cast<int4*>(a.seq + r0) = make_int4(seq[0], seq[1 % ROWS], seq[2 % ROWS], seq[3 % ROWS]);
        } else {
#pragma unroll
            for (int k = 0; k < ROWS; k++)
                if (at + k < a.rows) a.slots[r0 + k] = slot[k], a.pos[r0 + k] = pos[k], a.seq[r0 + k] = seq[k];
        }
    }
    // four pages given back at a time, a grid apart
    for (int64_t e0 = t; e0 < returned; e0 += 4 * nt) {
        int e[4], i[4], page[4];
#pragma unroll
        for (int k = 0; k < 4; k++) e[k] = (int)min(e0 + k * nt, (int64_t)returned - 1);
        last_le<4>(a.n, e, i, back);
#pragma unroll
        for (int k = 0; k < 4; k++) page[k] = __ldcg(a.table + (int64_t)i[k] * a.width + (e[k] - back(i[k])));
#pragma unroll
        for (int k = 0; k < 4; k++)
            if (e0 + k * nt < returned) a.free[wrap((unsigned)head + (unsigned)count + (unsigned)e[k], a.n_pages)] = page[k];  // (count + e < n_pages)
    }
}

// T threads.  FILL: both parts.
template <bool FILL, int T>
__global__ void __launch_bounds__(T) kv_pages_scan_kernel(PagesArgs a) {
    __shared__ int sm_start[FILL ? T : 1], sm_back[FILL ? T : 1];
    __shared__ int4 sm_request[FILL ? T : 1];
    __shared__ int sm_taken, sm_returned, sm_refused;
    const int t = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    int head = __ldcg(a.pool), count = __ldcg(a.pool + 1);
    if (t == 0) sm_taken = sm_returned = sm_refused = 0;
    int64_t before[3] = {0, 0, 0};  // rows, pages taken and pages given back by the requests before this round of T
    const int64_t most = (int64_t)a.width * a.page;
    for (int i0 = 0; i0 < a.n; i0 += T) {
        const int i = i0 + t;
        const bool in = i < a.n, live = i0 + (t & ~31) < a.n;
        const int len = in ? __ldcg(a.len + i) : 0, fresh = in ? __ldcg(a.fresh + i) : 0;
        if (i0 == 0) {
            head = head >= 0 && head < a.n_pages ? head : 0;
            count = min(max(count, 0), a.n_pages);
        }
        const bool ends = fresh < 0, sound = len >= 0 && len <= most;
        const int64_t grow = ends ? 0 : fresh, back = in && ends && sound ? pages_for(a, len) : 0;
        const int have = sound ? pages_for(a, len) : 0;
        bool fits = in && !ends && sound && len + grow <= most;
        int64_t need = fits ? pages_for(a, (int)(len + grow)) - have : 0, sums[3] = {grow, need, back}, total[3];
        cta_scan<T>(live, sums, total);
        if (before[0] + total[0] > a.rows) {  // some requests' rows do not fit: they take no pages
            if (before[0] + sums[0] > a.rows) fits = false, need = 0;
            sums[0] = grow, sums[1] = need, sums[2] = back;
            cta_scan<T>(live, sums, total);
        }
        const int64_t rows = before[0] + sums[0], taken = before[1] + sums[1], returned = before[2] + sums[2];
#pragma unroll
        for (int k = 0; k < 3; k++) before[k] += total[k];
        const bool served = fits && (need == 0 || taken <= count);
        const bool ended = in && ends && sound && (back == 0 || (int64_t)count + returned <= a.n_pages);
        if (in) {
            const int start = (int)clamp_int(rows - grow);
            const int4 q = make_int4(served ? (int)(need ? taken - need : 0) : ended ? kEnded : kRefused, len, have,
                                     (int)clamp_int(returned - back));
            a.start[i] = start;
            a.len_out[i] = served ? (int)(len + grow) : ended ? 0 : len;
            if (FILL)
                sm_start[i] = start, sm_back[i] = q.w, sm_request[i] = q;
            else
                a.ws[i] = q;
            if (served && need) atomicMax(&sm_taken, (int)taken);
            if (ended && back) atomicMax(&sm_returned, (int)returned);
            if (!served && !ended) atomicAdd(&sm_refused, 1);
        }
        __syncthreads();
    }
    const int total = (int)clamp_int(before[0]), taken = sm_taken, returned = sm_returned;
    if (t == 0) {
        a.start[a.n] = total;
        if (!FILL) a.ws[a.n] = make_int4(head, count, total, returned);
        a.pool_out[0] = wrap((unsigned)head + (unsigned)taken, a.n_pages);
        a.pool_out[1] = count - taken + returned;
        a.pool_out[2] = sm_refused;
        a.pool_out[3] = total;
    }
    if (FILL)
        fill<1>(a, t, T, total, returned, head, count, [&](int i) { return sm_start[i]; }, [&](int i) { return sm_back[i]; },
                [&](int i) { return sm_request[i]; });
}

// KEPT: the prefix sums in shared memory, so that the searches do not wait for L2.
template <bool KEPT>
__global__ void __launch_bounds__(kFill) kv_pages_fill_kernel(PagesArgs a) {
    extern __shared__ int sm_sums[];  // [n] starts, [n] pages given back
    pdl_launch_dependents();
    pdl_wait();
    const int4 h = __ldcg(a.ws + a.n);
    if (KEPT) {
        for (int i = threadIdx.x; i < a.n; i += kFill) sm_sums[i] = __ldcg(a.start + i), sm_sums[a.n + i] = __ldcg(&a.ws[i].w);
        __syncthreads();
    }
    const int64_t t = (int64_t)blockIdx.x * kFill + threadIdx.x, nt = (int64_t)gridDim.x * kFill;
    auto request = [&](int i) { return __ldcg(a.ws + i); };
    if (KEPT)
        fill<kFillRows>(a, t, nt, h.z, h.w, h.x, h.y, [&](int i) { return sm_sums[i]; }, [&](int i) { return sm_sums[a.n + i]; }, request);
    else
        fill<kFillRows>(a, t, nt, h.z, h.w, h.x, h.y, [&](int i) { return __ldcg(a.start + i); }, [&](int i) { return __ldcg(&a.ws[i].w); },
                        request);
}

}  // namespace

// One launch while a thread has few rows (64 requests with 704 rows 4.0 us, in two 6.3; with 2656 rows 7.3 in one and 6.2 in two, with
// 7856 15.6 and 6.3); in two, the sums in shared memory while they fit it beside 7 other CTAs' (7856 rows 6.3 us, without 7.4;
// 2000 requests 11.0 and 12.5).
cudaError_t launch_kv_pages(const PagesArgs& a, cudaStream_t s) {
    const bool few = a.n <= kFewSeqs;
    if (a.n <= kScan && a.rows <= 4 * (few ? kFewSeqs : kScan)) {
        if (few) return launch_chained(kv_pages_scan_kernel<true, kFewSeqs>, dim3(1), kFewSeqs, 0, s, a);
        return launch_chained(kv_pages_scan_kernel<true, kScan>, dim3(1), kScan, 0, s, a);
    }
    cudaError_t e = launch_chained(kv_pages_scan_kernel<false, kScan>, dim3(1), kScan, 0, s, a);
    if (e) return e;
    const int64_t work = std::max<int64_t>(a.rows, a.n);
    const int ctas = (int)std::min<int64_t>((work + kFill * kFillRows - 1) / (kFill * kFillRows), 8 * (int64_t)num_sms());
    if (a.n <= kKept) return launch_chained(kv_pages_fill_kernel<true>, dim3(std::max(ctas, 1)), kFill, 8 * a.n, s, a);
    return launch_chained(kv_pages_fill_kernel<false>, dim3(std::max(ctas, 1)), kFill, 0, s, a);
}

}  // namespace af

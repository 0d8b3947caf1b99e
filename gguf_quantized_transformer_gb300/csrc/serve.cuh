// Launchers of the operators of a serving step over a paged cache (pages and slots, paged attention, adapters).
#pragma once
#include "draft.cuh"

namespace af {

// ---- pages and slots (kv_pages.cu)
constexpr int kPagesMaxSeqs = 1 << 16;
struct PagesArgs {
    const int* len = nullptr;    // cached tokens of each request
    const int* fresh = nullptr;  // new tokens; negative: the request has ended
    int n = 0, page = 1, n_pages = 0, width = 0, rows = 0;
    const int* pool = nullptr;  // head and count of the ring of free pages
    int* free = nullptr;        // [n_pages]
    int* table = nullptr;       // [n][width]
    int* len_out = nullptr;
    int* pool_out = nullptr;
    int* start = nullptr;  // [n + 1]
    int *slots = nullptr, *pos = nullptr, *seq = nullptr;
    int4* ws = nullptr;  // [n + 1]
    unsigned page_mul = 0;  // position / page = umulhi(position, page_mul) >> page_shift; 0: page is 1
    int page_shift = 0;
    bool vec = false;  // slots, pos and seq are 16-byte aligned
};
cudaError_t launch_kv_pages(const PagesArgs& a, cudaStream_t s);

// ---- attention of single tokens over a paged cache (attn_paged.cu)
constexpr int kPagedMaxRows = 2048;
struct PagedArgs {
    const float* q = nullptr;
    int64_t ldq = 0;
    KvRows c;  // ctx = n_pages * page slots
    int H = 0, page = 1, n_pages = 0, width = 0, n_seqs = 0, n = 0;
    unsigned page_mul = 0;  // slot / page = umulhi(slot, page_mul) >> page_shift; 0: page is 1
    int page_shift = 0;
    bool wide = false;  // the stages of all rows and heads may pass 31 bits
    const int* table = nullptr;
    const int* seq = nullptr;  // nullable: row r is request r
    const int* pos = nullptr;
    float* out = nullptr;
    int64_t ldo = 0;
    float* ws = nullptr;
    unsigned long long mark = 0;  // 48 bits that a counter in a workspace of any contents does not hold
};
size_t attn_paged_ws_bytes(int D);
cudaError_t launch_attn_paged(const PagedArgs& a, cudaStream_t s);

// ---- low-rank adapters (lora.cu)
constexpr int kLoraMaxRows = 1 << 16, kLoraMaxAdapters = 4096, kLoraMaxRank = 128;
constexpr int kLoraTile = 32;  // rows of one adapter that a CTA takes at once
// A plan: header {tiles, tiles of adapters, rows of adapters, lora_plan_sizes}, the tiles {adapter or -1, first, count, 0}, then the
// rows in their order
__host__ __device__ constexpr int lora_plan_sizes(int n, int adapters) { return n | adapters << 17; }
static_assert(kLoraMaxRows < 1 << 17 && kLoraMaxAdapters < 1 << 13, "");
inline int lora_max_tiles(int n, int adapters) { return n / kLoraTile + (n < adapters + 1 ? n : adapters + 1); }
size_t lora_plan_bytes(int n, int adapters);
cudaError_t launch_lora_plan(const int* ids, int n, int adapters, void* plan, cudaStream_t s);
struct LoraArgs {
    const float* x = nullptr;
    int64_t ldx = 0;
    int n = 0;
    const void* plan = nullptr;
    const void *a = nullptr, *b = nullptr;  // [adapters][rank][K], [adapters][N][rank]
    int f16 = 0;
    const float* scale = nullptr;  // nullable
    const int* ranks = nullptr;    // nullable
    int adapters = 0, rank = 0, K = 0, N = 0;
    const float* base = nullptr;  // nullable: zeros
    int64_t ldb = 0;
    float* y = nullptr;
    int64_t ldy = 0;
    float* ws = nullptr;
};
size_t lora_ws_bytes(int n, int rank);
cudaError_t launch_lora(const LoraArgs& a, cudaStream_t s);

}  // namespace af

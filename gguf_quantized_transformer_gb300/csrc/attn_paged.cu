// Paged attention: the dispatch by cache type (attn_paged_impl.cuh).
#include <atomic>
#include <chrono>
#include <exception>
#include <random>

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

// A mark for the counters of one call.  A workspace may hold anything, so the counters do not start at a known number: what
// does not carry the call's mark counts as zero.  A call leaves each of its counters zero or with its mark and a count of zero,
// so that a captured one, whose mark is the same in every replay, finds them so.  The start is random: contents that this process did not write match with
// 2^-48.
unsigned long long next_mark() {
    static std::atomic<unsigned long long> at([] {
        unsigned long long seed = (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count();
        try {
            std::random_device r;
            seed ^= (unsigned long long)r() << 32 | r();
        } catch (const std::exception&) {  // (no source of randomness: the clock's count stands)
        }
        return seed * 0x9E3779B97F4A7C15ull;
    }());
    return at.fetch_add(0x9E3779B97F4Bull) & 0xFFFFFFFFFFFFull;
}

}  // namespace

size_t attn_paged_ws_bytes(int D) {
    return paged_ws_floats(num_sms(), D) * sizeof(float);
}

cudaError_t launch_attn_paged(const PagedArgs& args, cudaStream_t s) {
    PagedArgs a = args;
    // stages of 16 slots, of every row and head (a bound: tables as full as they can be)
    a.wide = ((int64_t)a.width * a.page / 16 + 1) * a.n > INT32_MAX / a.H;
    a.mark = next_mark();
    const int ctas = num_sms();
    switch (a.c.type) {
        case AF_F32: return launch_attn_paged_type<AF_F32>(a, ctas, s);
        case AF_F16: return launch_attn_paged_type<AF_F16>(a, ctas, s);
        case AF_KV_Q8_0: return launch_attn_paged_type<AF_KV_Q8_0>(a, ctas, s);
        default: return launch_attn_paged_type<AF_KV_Q4_0>(a, ctas, s);
    }
}

}  // namespace af

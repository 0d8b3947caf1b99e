#include "attn_paged_impl.cuh"

namespace af {
AF_PAGED_INSTANTIATE(AF_KV_Q8_0)
}  // namespace af

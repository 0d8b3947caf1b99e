#include "attn_paged_impl.cuh"

namespace af {
AF_PAGED_INSTANTIATE(AF_KV_Q4_0)
}  // namespace af

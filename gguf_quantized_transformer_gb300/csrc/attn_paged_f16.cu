#include "attn_paged_impl.cuh"

namespace af {
AF_PAGED_INSTANTIATE(AF_F16)
}  // namespace af

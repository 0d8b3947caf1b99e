#include "attn_paged_impl.cuh"

namespace af {
AF_PAGED_INSTANTIATE(AF_F32)
}  // namespace af

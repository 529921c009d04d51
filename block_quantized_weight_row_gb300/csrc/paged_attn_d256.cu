// paged_attn_d256.cu — the streaming paged-attention kernels for head_dim 256.
#include "paged_attn.cuh"

namespace bq {
namespace paged {
BQ_PAGED_STREAM_INSTANTIATE(8)
}  // namespace paged
}  // namespace bq

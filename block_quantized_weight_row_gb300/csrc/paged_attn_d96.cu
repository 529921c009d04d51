// paged_attn_d96.cu — the streaming paged-attention kernels for head_dim 96.
#include "paged_attn.cuh"

namespace bq {
namespace paged {
BQ_PAGED_STREAM_INSTANTIATE(3)
}  // namespace paged
}  // namespace bq

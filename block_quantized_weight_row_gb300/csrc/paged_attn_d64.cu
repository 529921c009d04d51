// paged_attn_d64.cu — the streaming paged-attention kernels for head_dim 64.
#include "paged_attn.cuh"

namespace bq {
namespace paged {
BQ_PAGED_STREAM_INSTANTIATE(2)
}  // namespace paged
}  // namespace bq

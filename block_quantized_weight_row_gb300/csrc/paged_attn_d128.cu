// paged_attn_d128.cu — the streaming paged-attention kernels for head_dim 128.
#include "paged_attn.cuh"

namespace bq {
namespace paged {
BQ_PAGED_STREAM_INSTANTIATE(4)
}  // namespace paged
}  // namespace bq

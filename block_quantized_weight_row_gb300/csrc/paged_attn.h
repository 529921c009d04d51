// paged_attn.h — what the host launchers and the kernels of the paged
// attention share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "paged.cuh"

namespace bq {

struct PagedAttnArgs {
  PagedPool kp, vp;
  PagedShape sh;
  const uint8_t *q;
  uint8_t *o;
  int64_t q_token, q_head, o_token, o_head;  // strides in bytes
  float *lse;                                // n_q x n_heads, or null
  const int32_t *q_start, *kv_len, *page_table;
  int64_t table_stride;
  int max_pages, n_seqs, n_q, max_kv, n_heads, group;
  int kt, vt, elem;
  float scale_log2;  // scale * log2(e): scores are kept in base-2 units
  int causal, window, rotate;
  // A sequence with more query rows (group * q_len) than this is the
  // tensor-memory kernel's, any other the streaming kernel's.
  int tc_rows;
  unsigned *err;
  // streaming kernel's partial results
  float *part_o;    // [cta][2][rows][D]
  float2 *part_ml;  // [cta][2][rows]: running maximum, sum of weights
  int4 *meta;       // [cta]: sequence, kv head, row group, last cta (or -1) of the split segment that starts there
  // many-row kernel's partial results, when its rows' tokens are split
  float *tc_part_o;    // [item][split][256][D]
  float2 *tc_part_ml;  // [item][split][256]
  int4 *tc_meta;       // [item]: sequence (or -1), kv head, first row, rows
};

// One sequence's lengths, checked: whatever the arrays hold, every row is in
// [0, n_q) and every token in [0, max_kv] and within the page table.
struct SeqSpan {
  int q0, q_len, kv;
};

__host__ __device__ __forceinline__ SeqSpan checked_span(int q0, int q1, int kv, int n_q, int64_t most_kv, bool &bad) {
  SeqSpan s{q0, q1 - q0, kv};
  bad = false;
  if (q0 < 0 || q1 < q0 || q1 > n_q) {
    s.q0 = s.q_len = 0;
    bad = true;
  }
  if (kv < 0 || kv > most_kv) {
    s.kv = kv < 0 ? 0 : int(most_kv);
    bad = true;
  }
  return s;
}

// Tokens [lo, hi) that query `i` of a sequence sees.
__host__ __device__ __forceinline__ void seen_range(const SeqSpan &s, int i, int causal, int window, int &lo, int &hi) {
  const int pos = s.kv - s.q_len + i;
  hi = causal ? (pos + 1 > 0 ? pos + 1 : 0) : s.kv;
  lo = (causal && window > 0 && pos - window + 1 > 0) ? pos - window + 1 : 0;
}

namespace paged {
// Shape of the streaming kernel (paged_attn.cuh) for head_dim 32 * NB, these
// cache types, and `rows8` groups of 8 query rows per kv head at most.
struct StreamShape {
  int rows, tokens, ctas_per_sm;  // rows per pass, tokens per tile
};
template <int NB>
StreamShape stream_shape(int kt, int vt, int elem, int rows8);
// beside: launched right after the many-row kernel of the same call
template <int NB>
cudaError_t launch_stream(const PagedAttnArgs &a, int rows8, int grid, int min_tiles, bool beside, cudaStream_t stream);

// The many-row kernel (paged_attn_tc.cu): `items` bounds the (kv head, 256
// rows) pairs of the sequences with more than tc_rows rows.
cudaError_t launch_tc(const PagedAttnArgs &a, int64_t items, int n_split, cudaStream_t stream);
}  // namespace paged

}  // namespace bq

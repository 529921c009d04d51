// layer.h — arguments of the kernels around the projections and the paged cache
// of a served layer (paged_extend.cu, norm.cu, rotary.cu, lora.cu). Sizes and
// pointers were checked by layer_api.cu; strides are in bytes.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bq {

struct ExtendArgs {
  const int32_t *kv_len, *n_new, *free_pages;
  int32_t *page_table, *q_start, *kv_out, *positions, *taken;
  int64_t *slots;
  int64_t max_pages;
  uint32_t page_size, n_pages, n_free, n_slots;
  uint32_t max_tokens;  // a sequence's longest length: the table's, and below 2^31
  int n_seqs;
  // set by the launcher:
  bool wide;            // slots and positions allow stores of two
  int page_shift;       // log2(page_size), or -1
  uint64_t page_magic;  // ceil(2^64 / (page_size / 16))
  unsigned *err;
};
cudaError_t launch_paged_extend(ExtendArgs a, cudaStream_t stream);

struct NormArgs {
  const uint8_t *x, *res;  // res: null for none
  uint8_t *sum, *out;      // null where not wanted
  uint8_t *q8;
  const float *weight;
  int64_t x_row, res_row, sum_row, out_row;
  int64_t n_rows;
  int n_cols;
  float inv_n[2], eps[2];  // each as a sum of two floats
};
cudaError_t launch_add_rms_norm(int elem, const NormArgs &a, cudaStream_t stream);

struct RotarySide {
  const uint8_t *in;
  uint8_t *out;
  int64_t in_token, in_head, out_token, out_head;
};
struct RotaryArgs {
  RotarySide side[2];  // q, k
  int heads[2];
  const int32_t *pos;
  int64_t pos_axis;  // elements between axes
  const double *inv_freq;
  const int32_t *axis;  // null: all 0
  int64_t n_tokens;
  int n_axes, dim, rot;
  bool interleaved, inverse;
  bool in_place;  // all outputs are their inputs: channels that no pair reaches need nothing
  bool onto;      // some output is its input
  unsigned *err;
};
cudaError_t launch_rotary(int elem_in, int elem_out, RotaryArgs a, cudaStream_t stream);

struct LoraArgs {
  const uint8_t *x, *A, *B, *y;  // y: null for none
  uint8_t *out;
  const float *scale;  // null: all 1
  const int32_t *adapter;
  int64_t x_row, y_row, out_row;
  int n_tokens, n_adapters, rank, K, M;
  bool y_vec;  // rows of y and out allow 16-byte accesses
  unsigned *err;
};
size_t lora_workspace_bytes(int64_t n_tokens, int64_t n_adapters, int64_t rank, int64_t K, int64_t M);
cudaError_t launch_lora(int x_elem, int w_elem, int y_elem, LoraArgs a, void *ws, cudaStream_t stream);

}  // namespace bq

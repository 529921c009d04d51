// layer_api.cu — the C ABI of the calls around the projections and the paged
// cache of a served layer (declared in include/bq.h): argument validation and
// the arguments the kernels take.
#include <algorithm>
#include <climits>

#include "bq.h"
#include "bq_device.cuh"
#include "bq_internal.h"
#include "layer.h"

namespace bq {
namespace {

int elem_bytes(int elem) { return elem == BQ_ELEM_F32 ? 4 : elem == BQ_ELEM_F16 || elem == BQ_ELEM_BF16 ? 2 : 0; }
bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// The bytes [p, p + n) of an argument; nothing where p is null.
struct Range {
  const void *p;
  uint64_t n;
};
bool meet(const Range &a, const Range &b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

// A range that is `steps` pieces, `step` bytes apart, of equal width. Two of them
// in one buffer (q and k of a fused projection) have spans that meet and pieces
// that do not: with the same step, pieces are compared modulo it.
struct Rows {
  Range r;
  int64_t step, steps;
};
bool meet(const Rows &a, const Rows &b) {
  if (!meet(a.r, b.r)) return false;
  if (a.step != b.step || a.step == 0) return true;
  const uint64_t step = uint64_t(a.step), wa = a.r.n - uint64_t(a.steps - 1) * step, wb = b.r.n - uint64_t(b.steps - 1) * step;
  if (wa > step || wb > step) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.r.p), y = reinterpret_cast<uintptr_t>(b.r.p);
  const uint64_t d = y >= x ? (y - x) % step : (step - (x - y) % step) % step;  // b's piece in a's step
  return d < wa || d + wb > step;
}

// Rows of `n` elements: their span of addresses, or the status of what is wrong.
int check_rows(const void *p, int64_t rows, int64_t n, int64_t stride, int es, uintptr_t align, const char *who, const char *name, Range &r) {
  if (!p) return report_error(BQ_ERR_INVALID_ARG, "%s: null %s", who, name);
  if (stride < 0 || stride > (int64_t(1) << 40)) return report_error(BQ_ERR_INVALID_ARG, "%s: the stride of %s is negative or above 2^40", who, name);
  if (!aligned(p, align) || (rows > 1 && uint64_t(stride) * es % align))
    return report_error(BQ_ERR_ALIGN, "%s: rows of %s must be %d-byte aligned", who, name, int(align));
  if ((double(rows - 1) * double(stride) + double(n)) * es > 4.0e18) return report_error(BQ_ERR_INVALID_ARG, "%s: %s spans too many bytes", who, name);
  r = Range{p, uint64_t((rows - 1) * stride + n) * es};
  return BQ_OK;
}

int launch_status(cudaError_t e, const char *who) {
  return e == cudaSuccess ? report_ok() : report_error(BQ_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
}

}  // namespace
}  // namespace bq

using namespace bq;

extern "C" {

int bq_paged_extend(int64_t page_size, int64_t n_pages, const int32_t *kv_len, const int32_t *n_new, int64_t n_seqs,
                    const int32_t *free_pages, int64_t n_free, int32_t *page_table, int64_t max_pages, int32_t *q_start,
                    int32_t *kv_len_out, int64_t *slots, int32_t *positions, int64_t n_slots, int32_t *taken) {
  const char *who = "bq_paged_extend";
  if (n_seqs < 0 || n_pages < 0 || n_free < 0 || max_pages < 0 || n_slots < 0 || page_size < 1)
    return report_error(BQ_ERR_INVALID_ARG, "%s: a size is negative", who);
  if (page_size % 16 || page_size > (1 << 20))
    return report_error(BQ_ERR_SHAPE, "%s: page_size %lld is not a multiple of 16 up to 2^20", who, (long long)page_size);
  if (n_pages > INT_MAX / page_size || n_seqs > (1 << 20) || n_slots > INT_MAX - 4096 || n_free > INT_MAX - 1 || max_pages > INT_MAX)
    return report_error(BQ_ERR_SHAPE, "%s: a size is above its limit (n_pages * page_size, n_slots, n_free 2^31, n_seqs 2^20)", who);
  if (!q_start || !taken || (n_slots > 0 && !slots) || (n_free > 0 && !free_pages))
    return report_error(BQ_ERR_INVALID_ARG, "%s: null pointer", who);
  if (n_seqs > 0 && (!kv_len || !n_new || !kv_len_out || (max_pages > 0 && !page_table)))
    return report_error(BQ_ERR_INVALID_ARG, "%s: null lengths or page table", who);
  if (!aligned(kv_len, 4) || !aligned(n_new, 4) || !aligned(free_pages, 4) || !aligned(page_table, 4) || !aligned(q_start, 4) ||
      !aligned(kv_len_out, 4) || !aligned(positions, 4) || !aligned(taken, 4) || !aligned(slots, 8))
    return report_error(BQ_ERR_ALIGN, "%s: int32 arguments must be 4-byte, slots 8-byte aligned", who);
  const uint64_t B = uint64_t(n_seqs) * 4;
  const Range ins[3] = {{kv_len, B}, {n_new, B}, {free_pages, uint64_t(n_free) * 4}};
  const Range outs[6] = {{page_table, B * uint64_t(max_pages)}, {q_start, B + 4}, {kv_len_out, B}, {slots, uint64_t(n_slots) * 8},
                         {positions, uint64_t(n_slots) * 4}, {taken, 8}};
  for (int i = 0; i < 6; ++i) {
    for (const Range &r : ins)
      if (meet(outs[i], r)) return report_error(BQ_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return report_error(BQ_ERR_INVALID_ARG, "%s: two outputs overlap", who);
  }
  ExtendArgs a{};
  a.kv_len = kv_len;
  a.n_new = n_new;
  a.free_pages = free_pages;
  a.page_table = page_table;
  a.q_start = q_start;
  a.kv_out = kv_len_out;
  a.positions = positions;
  a.taken = taken;
  a.slots = slots;
  a.max_pages = max_pages;
  a.page_size = uint32_t(page_size);
  a.n_pages = uint32_t(n_pages);
  a.n_free = uint32_t(n_free);
  a.n_slots = uint32_t(n_slots);
  a.max_tokens = uint32_t(std::min<int64_t>(max_pages * page_size, INT_MAX));
  a.n_seqs = int(n_seqs);
  return launch_status(launch_paged_extend(a, current_stream()), who);
}

int bq_add_rms_norm(int elem, const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                    const float *weight, double eps, void *sum, int64_t sum_stride, void *out, int64_t out_stride,
                    void *q8, int64_t n_rows, int64_t n_cols) {
  const char *who = "bq_add_rms_norm";
  const int es = elem_bytes(elem);
  if (!es) return report_error(BQ_ERR_UNSUPPORTED, "%s: unknown element type %d", who, elem);
  if (n_rows < 0 || n_cols < 0) return report_error(BQ_ERR_INVALID_ARG, "%s: a size is negative", who);
  if (n_cols % kQK || n_cols > BQ_RMS_NORM_MAX_COLS)
    return report_error(BQ_ERR_SHAPE, "%s: n_cols %lld is not a multiple of 32 up to %d", who, (long long)n_cols, BQ_RMS_NORM_MAX_COLS);
  if (n_rows > INT_MAX) return report_error(BQ_ERR_SHAPE, "%s: n_rows must be below 2^31", who);
  // what keeps the factor's arithmetic (m, 1 / m and the errors of both) among fp32's normal numbers
  if (!(eps >= 1e-30 && eps <= 1e30)) return report_error(BQ_ERR_INVALID_ARG, "%s: eps is not in 1e-30 .. 1e30", who);
  if (sum && !residual) return report_error(BQ_ERR_INVALID_ARG, "%s: a sum without a residual", who);
  if (!sum && !out && !q8) return report_error(BQ_ERR_INVALID_ARG, "%s: no output", who);
  if (n_rows == 0 || n_cols == 0) return report_ok();
  Range rx{}, rr{}, rs{}, ro{};
  int st;
  if ((st = check_rows(x, n_rows, n_cols, x_stride, es, 16, who, "x", rx)) != BQ_OK) return st;
  if (residual && (st = check_rows(residual, n_rows, n_cols, residual_stride, es, 16, who, "residual", rr)) != BQ_OK) return st;
  if (sum && (st = check_rows(sum, n_rows, n_cols, sum_stride, es, 16, who, "sum", rs)) != BQ_OK) return st;
  if (out && (st = check_rows(out, n_rows, n_cols, out_stride, es, 16, who, "out", ro)) != BQ_OK) return st;
  if (!weight) return report_error(BQ_ERR_INVALID_ARG, "%s: null weight", who);
  if (!aligned(weight, 16) || !aligned(q8, 16)) return report_error(BQ_ERR_ALIGN, "%s: weight and q8 must be 16-byte aligned", who);
  if (n_rows > 1 && ((sum && sum_stride < n_cols) || (out && out_stride < n_cols)))
    return report_error(BQ_ERR_INVALID_ARG, "%s: rows of an output overlap each other", who);
  const Range rw{weight, uint64_t(n_cols) * 4}, rq{q8, uint64_t(n_rows) * uint64_t(n_cols / kQK) * Fmt<kTypeQ8_0>::kBytes};
  const bool on_x = sum == x && (n_rows == 1 || sum_stride == x_stride), on_r = sum == residual && (n_rows == 1 || sum_stride == residual_stride);
  if ((meet(rs, rx) && !on_x) || (meet(rs, rr) && !on_r) || meet(rs, rw))
    return report_error(BQ_ERR_INVALID_ARG, "%s: sum overlaps an input that it is not", who);
  for (const Range &r : {ro, rq})
    if (meet(r, rx) || meet(r, rr) || meet(r, rw) || meet(r, rs)) return report_error(BQ_ERR_INVALID_ARG, "%s: an output overlaps another argument", who);
  if (meet(ro, rq)) return report_error(BQ_ERR_INVALID_ARG, "%s: two outputs overlap", who);
  NormArgs a{};
  a.x = static_cast<const uint8_t *>(x);
  a.res = static_cast<const uint8_t *>(residual);
  a.sum = static_cast<uint8_t *>(sum);
  a.out = static_cast<uint8_t *>(out);
  a.q8 = static_cast<uint8_t *>(q8);
  a.weight = weight;
  a.x_row = x_stride * es;
  a.res_row = residual_stride * es;
  a.sum_row = sum_stride * es;
  a.out_row = out_stride * es;
  a.n_rows = n_rows;
  a.n_cols = int(n_cols);
  const double inv = 1.0 / double(n_cols);
  a.inv_n[0] = float(inv);
  a.inv_n[1] = float(inv - a.inv_n[0]);
  a.eps[0] = float(eps);
  a.eps[1] = float(eps - a.eps[0]);
  return launch_status(launch_add_rms_norm(elem, a, current_stream()), who);
}

int bq_rotary(int elem, const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t n_q_heads, const void *k,
              int64_t k_token_stride, int64_t k_head_stride, int64_t n_k_heads, int elem_out, void *q_out,
              int64_t q_out_token_stride, int64_t q_out_head_stride, void *k_out, int64_t k_out_token_stride,
              int64_t k_out_head_stride, const int32_t *positions, int64_t position_stride, int64_t n_axes,
              const double *inv_freq, const int32_t *axis, int64_t rot, int64_t head_dim, int64_t n_tokens,
              int interleaved, int inverse) {
  const char *who = "bq_rotary";
  const int es = elem_bytes(elem), eo = elem_bytes(elem_out);
  if (!es || !eo || (elem != elem_out && elem != BQ_ELEM_F32))
    return report_error(BQ_ERR_UNSUPPORTED, "%s: element types %d to %d (the same, or from fp32)", who, elem, elem_out);
  if (n_q_heads < 0 || n_k_heads < 0 || n_tokens < 0 || rot < 0 || head_dim < 0)
    return report_error(BQ_ERR_INVALID_ARG, "%s: a size is negative", who);
  if (head_dim < kQK || head_dim % kQK || head_dim > 65536)
    return report_error(BQ_ERR_SHAPE, "%s: head_dim %lld is not a multiple of 32 up to 65536", who, (long long)head_dim);
  if (rot % 2 || rot > head_dim || rot > 16384)
    return report_error(BQ_ERR_SHAPE, "%s: rot %lld is odd or above head_dim or 16384", who, (long long)rot);
  if (n_axes < 1 || n_axes > BQ_ROTARY_MAX_AXES) return report_error(BQ_ERR_SHAPE, "%s: n_axes not in 1..%d", who, BQ_ROTARY_MAX_AXES);
  if (n_q_heads > 65536 || n_k_heads > 65536 || n_tokens > INT_MAX || (n_q_heads + n_k_heads) * head_dim > (1 << 24))
    return report_error(BQ_ERR_SHAPE, "%s: too many heads or tokens (channels of a token: 2^24)", who);
  if (n_tokens == 0 || n_q_heads + n_k_heads == 0) return report_ok();
  struct {
    const void *in;
    void *out;
    int64_t heads, it, ih, ot, oh;
    const char *name, *out_name;
  } t[2] = {{q, q_out, n_q_heads, q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride, "q", "q_out"},
            {k, k_out, n_k_heads, k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride, "k", "k_out"}};
  Range in[2] = {}, out[2] = {};
  bool same[2] = {true, true};
  RotaryArgs a{};
  for (int i = 0; i < 2; ++i) {
    if (t[i].heads == 0) continue;
    auto rows = [&](const void *p, int64_t ts, int64_t hs, int e, const char *name, Range &r) {
      if (!p) return report_error(BQ_ERR_INVALID_ARG, "%s: null %s", who, name);
      if (ts < 0 || hs < 0 || ts > (int64_t(1) << 40) || hs > (int64_t(1) << 40))
        return report_error(BQ_ERR_INVALID_ARG, "%s: a stride of %s is negative or above 2^40", who, name);
      if (!aligned(p, 16) || (n_tokens > 1 && ts * e % 16) || (t[i].heads > 1 && hs * e % 16))
        return report_error(BQ_ERR_ALIGN, "%s: rows of %s must be 16-byte aligned", who, name);
      if ((double(n_tokens - 1) * double(ts) + double(t[i].heads - 1) * double(hs) + double(head_dim)) * e > 4.0e18)
        return report_error(BQ_ERR_INVALID_ARG, "%s: %s spans too many bytes", who, name);
      r = Range{p, uint64_t((n_tokens - 1) * ts + (t[i].heads - 1) * hs + head_dim) * e};
      return BQ_OK;
    };
    int st;
    if ((st = rows(t[i].in, t[i].it, t[i].ih, es, t[i].name, in[i])) != BQ_OK) return st;
    if ((st = rows(t[i].out, t[i].ot, t[i].oh, eo, t[i].out_name, out[i])) != BQ_OK) return st;
    const bool by_token = (t[i].heads <= 1 || t[i].oh >= head_dim) && (n_tokens <= 1 || t[i].ot >= (t[i].heads - 1) * t[i].oh + head_dim);
    const bool by_head = (n_tokens <= 1 || t[i].ot >= head_dim) && (t[i].heads <= 1 || t[i].oh >= (n_tokens - 1) * t[i].ot + head_dim);
    if (!by_token && !by_head)
      return report_error(BQ_ERR_INVALID_ARG, "%s: rows of %s overlap each other", who, t[i].out_name);
    same[i] = t[i].in == t[i].out && elem == elem_out && (n_tokens <= 1 || t[i].it == t[i].ot) && (t[i].heads <= 1 || t[i].ih == t[i].oh);
    a.side[i] = RotarySide{static_cast<const uint8_t *>(t[i].in), static_cast<uint8_t *>(t[i].out), t[i].it * es, t[i].ih * es, t[i].ot * eo, t[i].oh * eo};
    a.heads[i] = int(t[i].heads);
  }
  if (rot > 0 && (!positions || !inv_freq)) return report_error(BQ_ERR_INVALID_ARG, "%s: null positions or frequencies", who);
  if (position_stride < 0 || position_stride > (int64_t(1) << 40)) return report_error(BQ_ERR_INVALID_ARG, "%s: bad position stride", who);
  if (!aligned(positions, 4) || !aligned(axis, 4) || !aligned(inv_freq, 8))
    return report_error(BQ_ERR_ALIGN, "%s: positions and axis must be 4-byte, inv_freq 8-byte aligned", who);
  const Range rest[3] = {{positions, uint64_t((n_axes - 1) * position_stride + n_tokens) * 4}, {inv_freq, uint64_t(rot / 2) * 8}, {axis, uint64_t(rot / 2) * 4}};
  const Rows ri[2] = {{in[0], t[0].it * es, n_tokens}, {in[1], t[1].it * es, n_tokens}};
  const Rows ro[2] = {{out[0], t[0].ot * eo, n_tokens}, {out[1], t[1].ot * eo, n_tokens}};
  if (meet(ro[0], ro[1])) return report_error(BQ_ERR_INVALID_ARG, "%s: the outputs overlap", who);
  for (int i = 0; i < 2; ++i) {
    for (int j = 0; j < 2; ++j)
      if (!(i == j && same[i]) && meet(ro[i], ri[j]))
        return report_error(BQ_ERR_INVALID_ARG, "%s: an output overlaps an input that it is not", who);
    for (const Range &r : rest)
      if (meet(out[i], r)) return report_error(BQ_ERR_INVALID_ARG, "%s: an output overlaps positions, frequencies or axes", who);
  }
  a.pos = positions;
  a.pos_axis = position_stride;
  a.inv_freq = inv_freq;
  a.axis = axis;
  a.n_tokens = n_tokens;
  a.n_axes = int(n_axes);
  a.dim = int(head_dim);
  a.rot = int(rot);
  a.interleaved = interleaved != 0;
  a.inverse = inverse != 0;
  a.in_place = same[0] && same[1];
  a.onto = (n_q_heads > 0 && same[0]) || (n_k_heads > 0 && same[1]);
  if (a.in_place && rot == 0) return report_ok();
  return launch_status(launch_rotary(elem, elem_out, a, current_stream()), who);
}

namespace {
int check_lora(int64_t n_tokens, int64_t n_adapters, int64_t rank, int64_t K, int64_t M, const char *who) {
  if (n_tokens < 0 || n_adapters < 0 || rank < 0 || K < 0 || M < 0) return report_error(BQ_ERR_INVALID_ARG, "%s: a size is negative", who);
  if (rank < 8 || rank % 8 || rank > BQ_LORA_MAX_RANK)
    return report_error(BQ_ERR_SHAPE, "%s: rank %lld is not a multiple of 8 up to %d", who, (long long)rank, BQ_LORA_MAX_RANK);
  if (K < kQK || K % kQK) return report_error(BQ_ERR_SHAPE, "%s: K %lld is not a multiple of 32", who, (long long)K);
  if (K >= (1 << 24) || M >= (1 << 24) || n_tokens > (1 << 20) || n_adapters > BQ_LORA_MAX_ADAPTERS)
    return report_error(BQ_ERR_SHAPE, "%s: a size is above its limit (K, M 2^24, n_tokens 2^20, n_adapters %d)", who, BQ_LORA_MAX_ADAPTERS);
  return BQ_OK;
}
}  // namespace

size_t bq_lora_workspace_size(int64_t n_tokens, int64_t n_adapters, int64_t rank, int64_t K, int64_t M) {
  if (check_lora(n_tokens, n_adapters, rank, K, M, "bq_lora_workspace_size") != BQ_OK || n_tokens == 0 || M == 0) return 0;
  return lora_workspace_bytes(n_tokens, n_adapters, rank, K, M);
}

int bq_lora(int x_elem, const void *x, int64_t x_stride, int w_elem, const void *A, const void *B, const float *scale,
            int64_t n_adapters, int64_t rank, const int32_t *adapter, int y_elem, const void *y, int64_t y_stride,
            void *out, int64_t out_stride, int64_t n_tokens, int64_t M, int64_t K) {
  const char *who = "bq_lora";
  const int xs = elem_bytes(x_elem), ys = elem_bytes(y_elem);
  if (w_elem != BQ_ELEM_F16 && w_elem != BQ_ELEM_BF16) return report_error(BQ_ERR_UNSUPPORTED, "%s: adapters are fp16 or bf16 (got type %d)", who, w_elem);
  if (!xs || !ys || (x_elem != BQ_ELEM_F32 && x_elem != w_elem) || (y_elem != BQ_ELEM_F32 && y_elem != w_elem))
    return report_error(BQ_ERR_UNSUPPORTED, "%s: x and y are fp32 or of the adapters' type (got %d, %d beside %d)", who, x_elem, y_elem, w_elem);
  int st = check_lora(n_tokens, n_adapters, rank, K, M, who);
  if (st != BQ_OK) return st;
  if (n_tokens == 0 || M == 0) return report_ok();
  Range rx{}, ry{}, ro{};
  if ((st = check_rows(x, n_tokens, K, x_stride, xs, 16, who, "x", rx)) != BQ_OK) return st;
  if (y && (st = check_rows(y, n_tokens, M, y_stride, ys, ys, who, "y", ry)) != BQ_OK) return st;
  if ((st = check_rows(out, n_tokens, M, out_stride, ys, ys, who, "out", ro)) != BQ_OK) return st;
  if (n_tokens > 1 && out_stride < M) return report_error(BQ_ERR_INVALID_ARG, "%s: rows of out overlap each other", who);
  if (!adapter || (n_adapters > 0 && (!A || !B))) return report_error(BQ_ERR_INVALID_ARG, "%s: null adapters", who);
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(scale, 4) || !aligned(adapter, 4))
    return report_error(BQ_ERR_ALIGN, "%s: A and B must be 16-byte, scale and adapter 4-byte aligned", who);
  const Range ins[5] = {rx, {A, uint64_t(n_adapters) * uint64_t(rank * K) * 2}, {B, uint64_t(n_adapters) * uint64_t(rank * M) * 2},
                        {scale, uint64_t(n_adapters) * 4}, {adapter, uint64_t(n_tokens) * 4}};
  for (const Range &r : ins)
    if (meet(ro, r)) return report_error(BQ_ERR_INVALID_ARG, "%s: out overlaps an input", who);
  if (meet(ro, ry) && !(y == out && (n_tokens == 1 || y_stride == out_stride)))
    return report_error(BQ_ERR_INVALID_ARG, "%s: out overlaps y without being it", who);
  size_t ws_bytes;
  void *ws = current_workspace(&ws_bytes);
  const size_t need = lora_workspace_bytes(n_tokens, n_adapters, rank, K, M);
  if (!ws || ws_bytes < need) return report_error(BQ_ERR_WORKSPACE, "%s: needs %zu workspace bytes, %zu set", who, need, ws_bytes);
  const Range rw{ws, need};
  for (const Range &r : ins)
    if (meet(rw, r)) return report_error(BQ_ERR_INVALID_ARG, "%s: the workspace overlaps an argument", who);
  if (meet(rw, ry) || meet(rw, ro)) return report_error(BQ_ERR_INVALID_ARG, "%s: the workspace overlaps an argument", who);
  LoraArgs a{};
  a.x = static_cast<const uint8_t *>(x);
  a.A = static_cast<const uint8_t *>(A);
  a.B = static_cast<const uint8_t *>(B);
  a.y = static_cast<const uint8_t *>(y);
  a.out = static_cast<uint8_t *>(out);
  a.scale = scale;
  a.adapter = adapter;
  a.x_row = x_stride * xs;
  a.y_row = y_stride * ys;
  a.out_row = out_stride * ys;
  a.n_tokens = int(n_tokens);
  a.n_adapters = int(n_adapters);
  a.rank = int(rank);
  a.K = int(K);
  a.M = int(M);
  const bool one = n_tokens == 1;
  a.y_vec = aligned(out, 16) && (one || a.out_row % 16 == 0) && (!y || (aligned(y, 16) && (one || a.y_row % 16 == 0)));
  return launch_status(launch_lora(x_elem, w_elem, y_elem, a, ws, current_stream()), who);
}

}  // extern "C"

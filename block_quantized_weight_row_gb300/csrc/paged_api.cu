// paged_api.cu — the C ABI of the paged KV cache (declared in include/bq.h):
// argument validation and the descriptors the kernels take.
#include <algorithm>
#include <climits>
#include <cmath>

#include "bq.h"
#include "bq_device.cuh"
#include "bq_internal.h"
#include "paged_attn.h"

namespace bq {
namespace {

bool core(int type) { return type == BQ_TYPE_Q4_0 || type == BQ_TYPE_Q8_0; }
int block_size(int type) { return type == BQ_TYPE_Q4_0 ? Fmt<kTypeQ4_0>::kBytes : Fmt<kTypeQ8_0>::kBytes; }
int code_size(int type) { return type == BQ_TYPE_Q4_0 ? Codes<kTypeQ4_0>::kBytes : Codes<kTypeQ8_0>::kBytes; }
bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// [a, a + na) and [b, b + nb) share a byte
bool meet(const void *a, uint64_t na, const void *b, uint64_t nb) {
  if (!a || !b || !na || !nb) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

struct Range {
  const void *p;
  uint64_t n;
};

struct Cache {
  PagedShape sh;
  PagedPool k, v;
  uint64_t k_bytes, v_bytes;
};

// The descriptor of a cache, or the status of what is wrong with it.
int check_cache(const bq_paged_cache *c, const char *who, Cache &out) {
  if (!c) return report_error(BQ_ERR_INVALID_ARG, "%s: null cache", who);
  if (!core(c->k_type) || !core(c->v_type))
    return report_error(BQ_ERR_UNSUPPORTED, "%s: K and V types must be Q4_0 or Q8_0 (got %d, %d)", who, c->k_type, c->v_type);
  if (c->k_basis != BQ_BASIS_PLAIN && c->k_basis != BQ_BASIS_HADAMARD64)
    return report_error(BQ_ERR_UNSUPPORTED, "%s: unknown basis %d", who, c->k_basis);
  if (c->n_pages < 0 || c->n_kv_heads < 1 || c->head_dim < 1 || c->page_size < 1)
    return report_error(BQ_ERR_INVALID_ARG, "%s: bad cache sizes", who);
  if (c->page_size % kPagedTile || c->page_size > (1 << 20))
    return report_error(BQ_ERR_SHAPE, "%s: page_size %lld is not a multiple of %d up to 2^20", who, (long long)c->page_size, kPagedTile);
  if (c->head_dim % kQK || c->head_dim > 65536)
    return report_error(BQ_ERR_SHAPE, "%s: head_dim %lld is not a multiple of 32 up to 65536", who, (long long)c->head_dim);
  if (c->k_basis == BQ_BASIS_HADAMARD64 && c->head_dim % 64)
    return report_error(BQ_ERR_SHAPE, "%s: the rotated basis needs head_dim %% 64 == 0", who);
  if (c->n_kv_heads > 65536 || c->n_kv_heads * (c->head_dim / kQK) > (1 << 20))
    return report_error(BQ_ERR_SHAPE, "%s: n_kv_heads above 2^16 or n_kv_heads * head_dim above 2^25", who);
  if (c->n_pages > INT_MAX / c->page_size)
    return report_error(BQ_ERR_SHAPE, "%s: n_pages * page_size must be below 2^31 tokens", who);
  if (c->n_pages > 0 && (!c->k_pages || !c->v_pages)) return report_error(BQ_ERR_INVALID_ARG, "%s: null page pool", who);
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16))
    return report_error(BQ_ERR_ALIGN, "%s: page pools must be 16-byte aligned", who);
  const int nb = int(c->head_dim / kQK);
  int shift = -1;
  if ((c->page_size & (c->page_size - 1)) == 0)
    for (shift = 0; (int64_t(1) << shift) < c->page_size;) ++shift;
  const uint64_t p16 = uint64_t(c->page_size / kPagedTile);
  out.sh = PagedShape{c->n_pages, int(c->page_size), shift, ~uint64_t(0) / p16 + 1, int(c->n_kv_heads), nb};
  auto pool = [&](void *base, int type) {
    PagedPool p;
    p.base = static_cast<uint8_t *>(base);
    p.row_bytes = nb * code_size(type);
    p.scale_off = c->page_size * p.row_bytes;
    p.head_bytes = c->page_size * nb * block_size(type);
    return p;
  };
  out.k = pool(c->k_pages, c->k_type);
  out.v = pool(c->v_pages, c->v_type);
  out.k_bytes = uint64_t(c->n_pages) * uint64_t(c->n_kv_heads) * uint64_t(out.k.head_bytes);
  out.v_bytes = uint64_t(c->n_pages) * uint64_t(c->n_kv_heads) * uint64_t(out.v.head_bytes);
  if (meet(c->k_pages, out.k_bytes, c->v_pages, out.v_bytes))
    return report_error(BQ_ERR_INVALID_ARG, "%s: the K and V pools overlap", who);
  return BQ_OK;
}

int elem_bytes(int elem) { return elem == BQ_ELEM_F32 ? 4 : elem == BQ_ELEM_F16 || elem == BQ_ELEM_BF16 ? 2 : 0; }

int check_bias(const bq_paged_cache *c, const float *bias, int bias_basis, const char *who) {
  if (!bias) return BQ_OK;
  if (c->k_type != BQ_TYPE_Q4_0)
    return report_error(BQ_ERR_UNSUPPORTED, "%s: a mean-centering bias requires a Q4_0 K cache", who);
  if (bias_basis != c->k_basis)
    return report_error(BQ_ERR_BASIS, "%s: the bias was calibrated in basis %d, the cache is in basis %d", who, bias_basis, c->k_basis);
  if (!aligned(bias, 16)) return report_error(BQ_ERR_ALIGN, "%s: bias must be 16-byte aligned", who);
  return BQ_OK;
}

// A strided [token][head][head_dim] tensor of 16-byte aligned rows. `bytes`:
// the span of its addresses.
int check_rows(const void *p, int64_t n_tokens, int64_t heads, int64_t D, int64_t ts, int64_t hs, int es, const char *who,
               const char *name, uint64_t &bytes) {
  if (!p) return report_error(BQ_ERR_INVALID_ARG, "%s: null %s", who, name);
  if (ts < 0 || hs < 0 || ts > (int64_t(1) << 40) || hs > (int64_t(1) << 40))
    return report_error(BQ_ERR_INVALID_ARG, "%s: a stride of %s is negative or above 2^40", who, name);
  if (!aligned(p, 16) || (n_tokens > 1 && ts * es % 16) || (heads > 1 && hs * es % 16))
    return report_error(BQ_ERR_ALIGN, "%s: rows of %s must be 16-byte aligned", who, name);
  // counts below 2^31 times strides up to 2^40: judged in floating point before the 64-bit product
  const double span = (double(n_tokens - 1) * double(ts) + double(heads - 1) * double(hs) + double(D)) * es;
  if (span > 4.0e18) return report_error(BQ_ERR_INVALID_ARG, "%s: %s spans too many bytes", who, name);
  bytes = uint64_t(((n_tokens - 1) * ts + (heads - 1) * hs + D) * es);
  return BQ_OK;
}

// Rows that are written must not share elements: heads within a token, or
// tokens within a head, lie apart by whole rows.
bool rows_distinct(int64_t n_tokens, int64_t heads, int64_t D, int64_t ts, int64_t hs) {
  const bool by_token = (heads <= 1 || hs >= D) && (n_tokens <= 1 || ts >= (heads - 1) * hs + D);
  const bool by_head = (n_tokens <= 1 || ts >= D) && (heads <= 1 || hs >= (n_tokens - 1) * ts + D);
  return by_token || by_head;
}

// The sizes of an attention call, into the kernels' arguments.
int check_attn(const bq_paged_cache *cache, int elem, int64_t n_seqs, int64_t n_q, int64_t max_q, int64_t max_kv,
               int64_t max_pages, int64_t n_heads, int causal, int64_t window, const char *who, Cache &c, PagedAttnArgs &a) {
  const int st = check_cache(cache, who, c);
  if (st != BQ_OK) return st;
  if (!elem_bytes(elem)) return report_error(BQ_ERR_UNSUPPORTED, "%s: unknown element type %d", who, elem);
  if (!paged_attn_dim(cache->head_dim))
    return report_error(BQ_ERR_SHAPE, "%s: head_dim %lld is not 64, 96, 128 or 256", who, (long long)cache->head_dim);
  if (n_seqs < 0 || n_q < 0 || max_q < 0 || max_kv < 0 || max_pages < 0 || window < 0)
    return report_error(BQ_ERR_INVALID_ARG, "%s: a size is negative", who);
  if (n_heads < 1 || n_heads > 65536 || n_heads % cache->n_kv_heads)
    return report_error(BQ_ERR_SHAPE, "%s: n_heads %lld is not a multiple of n_kv_heads up to 65536", who, (long long)n_heads);
  if (n_seqs > (1 << 20) || max_kv > INT_MAX - 65536 || max_pages > INT_MAX || n_q > INT_MAX / 2 ||
      n_q * (n_heads / cache->n_kv_heads) > INT_MAX / 2)
    return report_error(BQ_ERR_SHAPE, "%s: a size is above its limit (n_seqs 2^20, n_q * n_heads / n_kv_heads 2^30)", who);
  if (window > 0 && !causal) return report_error(BQ_ERR_UNSUPPORTED, "%s: a window needs causal attention", who);
  a = PagedAttnArgs{};
  a.kp = c.k;
  a.vp = c.v;
  a.sh = c.sh;
  a.max_pages = int(max_pages);
  a.n_seqs = int(n_seqs);
  a.n_q = int(n_q);
  a.max_kv = int(max_kv);
  a.n_heads = int(n_heads);
  a.group = int(n_heads / cache->n_kv_heads);
  a.kt = cache->k_type;
  a.vt = cache->v_type;
  a.elem = elem;
  a.causal = causal != 0;
  a.window = int(window > INT_MAX / 2 ? INT_MAX / 2 : window);
  a.rotate = cache->k_basis == BQ_BASIS_HADAMARD64;
  a.tc_rows = INT_MAX;
  return BQ_OK;
}

}  // namespace
}  // namespace bq

using namespace bq;

extern "C" {

size_t bq_paged_page_bytes(int type, int64_t page_size, int64_t n_kv_heads, int64_t head_dim) {
  if (!core(type) || page_size < 1 || page_size % kPagedTile || page_size > (1 << 20) || n_kv_heads < 1 ||
      n_kv_heads > 65536 || head_dim < kQK || head_dim % kQK || head_dim > 65536)
    return 0;
  return size_t(page_size) * size_t(n_kv_heads) * size_t(head_dim / kQK) * size_t(block_size(type));
}

int bq_paged_kv_write(const bq_paged_cache *cache, int elem, const void *K, int64_t k_token_stride,
                      int64_t k_head_stride, const void *V, int64_t v_token_stride, int64_t v_head_stride,
                      const float *bias, int bias_basis, const int64_t *slots, int64_t n_tokens) {
  const char *who = "bq_paged_kv_write";
  Cache c;
  int st = check_cache(cache, who, c);
  if (st != BQ_OK) return st;
  const int es = elem_bytes(elem);
  if (!es) return report_error(BQ_ERR_UNSUPPORTED, "%s: unknown element type %d", who, elem);
  if ((st = check_bias(cache, bias, bias_basis, who)) != BQ_OK) return st;
  if (n_tokens < 0 || n_tokens > INT_MAX) return report_error(BQ_ERR_INVALID_ARG, "%s: bad token count", who);
  if (n_tokens == 0) return report_ok();
  const int64_t H = cache->n_kv_heads, D = cache->head_dim;
  uint64_t kb, vb;
  if ((st = check_rows(K, n_tokens, H, D, k_token_stride, k_head_stride, es, who, "K", kb)) != BQ_OK) return st;
  if ((st = check_rows(V, n_tokens, H, D, v_token_stride, v_head_stride, es, who, "V", vb)) != BQ_OK) return st;
  if (!slots) return report_error(BQ_ERR_INVALID_ARG, "%s: null slots", who);
  if (!aligned(slots, 8)) return report_error(BQ_ERR_ALIGN, "%s: slots must be 8-byte aligned", who);
  const Range pools[2] = {{cache->k_pages, c.k_bytes}, {cache->v_pages, c.v_bytes}};
  for (const Range &p : pools)
    if (meet(p.p, p.n, K, kb) || meet(p.p, p.n, V, vb) || meet(p.p, p.n, bias, uint64_t(H * D) * 4) ||
        meet(p.p, p.n, slots, uint64_t(n_tokens) * 8))
      return report_error(BQ_ERR_INVALID_ARG, "%s: a page pool overlaps an input", who);
  const cudaError_t e = launch_paged_write(c.k, c.v, c.sh, cache->k_type, cache->v_type, elem, cache->k_basis == BQ_BASIS_HADAMARD64,
                                           K, k_token_stride * es, k_head_stride * es, V, v_token_stride * es, v_head_stride * es,
                                           bias, slots, n_tokens, current_stream());
  return e == cudaSuccess ? report_ok() : report_error(BQ_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
}

int bq_paged_kv_read(const bq_paged_cache *cache, int elem, void *K, void *V, const float *bias, int bias_basis,
                     const int64_t *slots, int64_t n_tokens) {
  const char *who = "bq_paged_kv_read";
  Cache c;
  int st = check_cache(cache, who, c);
  if (st != BQ_OK) return st;
  const int es = elem_bytes(elem);
  if (!es) return report_error(BQ_ERR_UNSUPPORTED, "%s: unknown element type %d", who, elem);
  if ((st = check_bias(cache, bias, bias_basis, who)) != BQ_OK) return st;
  if (n_tokens < 0 || n_tokens > INT_MAX) return report_error(BQ_ERR_INVALID_ARG, "%s: bad token count", who);
  if (n_tokens == 0) return report_ok();
  const int64_t H = cache->n_kv_heads, D = cache->head_dim;
  if (!K || !V || !slots) return report_error(BQ_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 8))
    return report_error(BQ_ERR_ALIGN, "%s: K and V must be 16-byte, slots 8-byte aligned", who);
  if (cache->n_pages == 0) return report_error(BQ_ERR_INVALID_ARG, "%s: the cache has no pages", who);
  const uint64_t out = uint64_t(n_tokens) * uint64_t(H * D) * uint64_t(es);
  const Range ins[4] = {{cache->k_pages, c.k_bytes}, {cache->v_pages, c.v_bytes}, {bias, uint64_t(H * D) * 4}, {slots, uint64_t(n_tokens) * 8}};
  for (const Range &p : ins)
    if (meet(p.p, p.n, K, out) || meet(p.p, p.n, V, out))
      return report_error(BQ_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
  if (meet(K, out, V, out)) return report_error(BQ_ERR_INVALID_ARG, "%s: the outputs overlap", who);
  const cudaError_t e = launch_paged_read(c.k, c.v, c.sh, cache->k_type, cache->v_type, elem, cache->k_basis == BQ_BASIS_HADAMARD64,
                                          K, V, bias, slots, n_tokens, current_stream());
  return e == cudaSuccess ? report_ok() : report_error(BQ_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
}

size_t bq_paged_attn_workspace_size(const bq_paged_cache *cache, int elem, int64_t n_seqs, int64_t n_q, int64_t max_q_len,
                                    int64_t max_kv_len, int64_t n_heads, int causal, int64_t window) {
  Cache c;
  PagedAttnArgs a;
  if (check_attn(cache, elem, n_seqs, n_q, max_q_len, max_kv_len, 0, n_heads, causal, window, "bq_paged_attn_workspace_size", c, a) != BQ_OK)
    return 0;
  return paged_attn_workspace_bytes(a, int(std::min(max_q_len, n_q)));
}

int64_t bq_paged_attn_many_rows(const bq_paged_cache *cache, int elem, int64_t n_seqs, int64_t n_q, int64_t max_q_len,
                                int64_t max_kv_len, int64_t n_heads, int causal, int64_t window) {
  Cache c;
  PagedAttnArgs a;
  if (check_attn(cache, elem, n_seqs, n_q, max_q_len, max_kv_len, 0, n_heads, causal, window, "bq_paged_attn_many_rows", c, a) != BQ_OK)
    return 0;
  return paged_attn_many_rows(a, int(std::min(max_q_len, n_q)));
}

int bq_paged_attn(const bq_paged_cache *cache, int elem, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                  void *o, int64_t o_token_stride, int64_t o_head_stride, float *lse, const int32_t *q_start,
                  const int32_t *kv_len, const int32_t *page_table, int64_t max_pages, int64_t n_seqs, int64_t n_q,
                  int64_t max_q_len, int64_t max_kv_len, int64_t n_heads, float scale, int causal, int64_t window) {
  const char *who = "bq_paged_attn";
  Cache c;
  PagedAttnArgs a;
  int st = check_attn(cache, elem, n_seqs, n_q, max_q_len, max_kv_len, max_pages, n_heads, causal, window, who, c, a);
  if (st != BQ_OK) return st;
  if (!std::isfinite(scale)) return report_error(BQ_ERR_INVALID_ARG, "%s: scale is not finite", who);
  if (n_seqs == 0 || n_q == 0) return report_ok();
  if (cache->n_pages == 0) return report_error(BQ_ERR_INVALID_ARG, "%s: the cache has no pages", who);
  const int64_t D = cache->head_dim;
  const int es = elem_bytes(elem);
  uint64_t qb, ob;
  if ((st = check_rows(q, n_q, n_heads, D, q_token_stride, q_head_stride, es, who, "q", qb)) != BQ_OK) return st;
  if ((st = check_rows(o, n_q, n_heads, D, o_token_stride, o_head_stride, es, who, "o", ob)) != BQ_OK) return st;
  if (!rows_distinct(n_q, n_heads, D, o_token_stride, o_head_stride))
    return report_error(BQ_ERR_INVALID_ARG, "%s: rows of o overlap each other", who);
  if (!q_start || !kv_len || (!page_table && max_pages > 0)) return report_error(BQ_ERR_INVALID_ARG, "%s: null lengths or page table", who);
  if (!aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4) || !aligned(lse, 4))
    return report_error(BQ_ERR_ALIGN, "%s: lengths, page table and lse must be 4-byte aligned", who);
  const uint64_t lb = lse ? uint64_t(n_q) * uint64_t(n_heads) * 4 : 0;
  size_t ws_bytes;
  void *ws = current_workspace(&ws_bytes);
  const int max_q = int(std::min(max_q_len, n_q));
  const size_t need = paged_attn_workspace_bytes(a, max_q);
  const Range ins[6] = {{cache->k_pages, c.k_bytes}, {cache->v_pages, c.v_bytes}, {q, qb},
                        {q_start, uint64_t(n_seqs + 1) * 4}, {kv_len, uint64_t(n_seqs) * 4},
                        {page_table, uint64_t(n_seqs) * uint64_t(max_pages) * 4}};
  for (const Range &p : ins)
    if (meet(p.p, p.n, o, ob) || meet(p.p, p.n, lse, lb))
      return report_error(BQ_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
  if (meet(o, ob, lse, lb)) return report_error(BQ_ERR_INVALID_ARG, "%s: o and lse overlap", who);
  if (!ws || ws_bytes < need)
    return report_error(BQ_ERR_WORKSPACE, "%s: needs %zu workspace bytes, %zu set", who, need, ws_bytes);
  for (const Range &p : ins)
    if (meet(p.p, p.n, ws, need)) return report_error(BQ_ERR_INVALID_ARG, "%s: the workspace overlaps an input", who);
  if (meet(o, ob, ws, need) || meet(lse, lb, ws, need))
    return report_error(BQ_ERR_INVALID_ARG, "%s: the workspace overlaps an output", who);
  a.q = static_cast<const uint8_t *>(q);
  a.o = static_cast<uint8_t *>(o);
  a.q_token = q_token_stride * es;
  a.q_head = q_head_stride * es;
  a.o_token = o_token_stride * es;
  a.o_head = o_head_stride * es;
  a.lse = lse;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.table_stride = max_pages;
  a.scale_log2 = scale * 1.4426950408889634f;
  const cudaError_t e = launch_paged_attn(a, max_q, ws, current_stream());
  return e == cudaSuccess ? report_ok() : report_error(BQ_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
}

int bq_paged_slot_check(const bq_paged_cache *cache, int64_t slot, int64_t *page, int64_t *place) {
  Cache c;
  const int st = check_cache(cache, "bq_paged_slot_check", c);
  if (st != BQ_OK) return st;
  if (!page || !place) return report_error(BQ_ERR_INVALID_ARG, "bq_paged_slot_check: null pointer");
  *page = *place = -1;
  switch (slot_kind(c.sh, slot)) {
    case SlotKind::kSkip: return report_ok();
    case SlotKind::kBad: return report_error(BQ_ERR_INDEX, "bq_paged_slot_check: slot %lld is outside the pool", (long long)slot);
    default: break;
  }
  uint32_t p, i;
  split_slot(c.sh, uint32_t(slot), p, i);
  *page = p;
  *place = i;
  return report_ok();
}

}  // extern "C"

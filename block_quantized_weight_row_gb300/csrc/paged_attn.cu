// paged_attn.cu — paged attention: the combine of split segments, the choice
// of kernel and grid, and the workspace.
#include <algorithm>

#include "paged_attn.cuh"

namespace bq {
namespace {

using paged::StreamShape;

constexpr int kMaxSms = 160;           // the workspace is sized without asking the device
constexpr int kMaxCtas = 2 * kMaxSms;  // pieces of the streaming kernel at most
constexpr int kCombineThreads = 256;

// Merges partial results. Blocks below grid * rows take one row of one split
// segment of the streaming kernel: block (i, r) the segment that starts in
// piece i, if there is one, and its row r; 256 threads read several partials
// at a time, D / 4 threads per row. The blocks after them take 1024 / D rows
// each of the many-row kernel's items. Bound by latency: at most a few
// megabytes come out of L2. The order of the sums is fixed.
__global__ void __launch_bounds__(kCombineThreads)
    k_paged_combine(const __grid_constant__ PagedAttnArgs a, int grid, int rows, int D, int n_split) {
  __shared__ float weight[kMaxCtas];
  __shared__ float red[kCombineThreads / 32][2];
  __shared__ float4 acc_s[kCombineThreads];
  const int quads = D / 4, per = kCombineThreads / quads;
  const int ch = int(threadIdx.x) % quads * 4, k = int(threadIdx.x) / quads, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  auto finish = [&](const SeqSpan &span, int kvh, int row, float4 acc, float top, float sum) {
    const int tok = row / a.group, head = kvh * a.group + (row - tok * a.group);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint8_t *out = a.o + int64_t(span.q0 + tok) * a.o_token + int64_t(head) * a.o_head;
    paged::store_out4(a.elem, out, ch, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (ch == 0 && a.lse)
      a.lse[int64_t(span.q0 + tok) * a.n_heads + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / paged::kLog2e;
  };
  if (int(blockIdx.x) >= grid * rows) {
    const int blocks = (256 + per - 1) / per, i = int(blockIdx.x) - grid * rows, item = i / blocks, r = (i - item * blocks) * per + k;
    const int4 mt = a.tc_meta[item];
    if (mt.x < 0 || k >= per || r >= mt.w) return;
    const int64_t p0 = int64_t(item) * n_split * 256 + r;
    float top = -INFINITY, sum = 0.0f;
    for (int s = 0; s < n_split; ++s) top = fmaxf(top, a.tc_part_ml[p0 + s * 256].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < n_split; ++s) {
      const float2 ml = a.tc_part_ml[p0 + s * 256];
      if (ml.y == 0.0f) continue;
      const float w = paged::ex2(ml.x - top);
      const float4 v = *reinterpret_cast<const float4 *>(a.tc_part_o + (p0 + s * 256) * D + ch);
      sum = fmaf(ml.y, w, sum);
      acc.x = fmaf(v.x, w, acc.x), acc.y = fmaf(v.y, w, acc.y), acc.z = fmaf(v.z, w, acc.z), acc.w = fmaf(v.w, w, acc.w);
    }
    finish(paged::load_span(a, mt.x, false), mt.y, mt.z + r, acc, top, sum);
    return;
  }
  const int first = int(blockIdx.x) / rows, r = int(blockIdx.x) - first * rows;
  const int4 mt = a.meta[first];
  if (mt.w < 0) return;
  const SeqSpan span = paged::load_span(a, mt.x, false);
  const int row = mt.z * rows + r;
  if (row >= span.q_len * a.group) return;
  const int n = mt.w - first + 1;
  auto part = [&](int i) { return (int64_t(first + i) * 2 + (i == 0 ? 1 : 0)) * rows + r; };
  float top = paged::kNoMax;
  for (int i = threadIdx.x; i < n; i += kCombineThreads) top = fmaxf(top, a.part_ml[part(i)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  if (lane == 0) red[warp][0] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCombineThreads / 32; ++w) top = fmaxf(top, red[w][0]);
  float sum = 0.0f;
  for (int i = threadIdx.x; i < n; i += kCombineThreads) {
    const float2 ml = a.part_ml[part(i)];
    const float w = ml.y == 0.0f ? 0.0f : paged::ex2(ml.x - top);
    weight[i] = w;
    sum = fmaf(ml.y, w, sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) red[warp][1] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kCombineThreads / 32; ++w) sum += red[w][1];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = k; i < n && k < per; i += per) {
    const float w = weight[i];
    if (w == 0.0f) continue;  // nothing was seen there
    const float4 v = *reinterpret_cast<const float4 *>(a.part_o + part(i) * D + ch);
    acc.x = fmaf(v.x, w, acc.x), acc.y = fmaf(v.y, w, acc.y), acc.z = fmaf(v.z, w, acc.z), acc.w = fmaf(v.w, w, acc.w);
  }
  acc_s[threadIdx.x] = acc;
  __syncthreads();
  if (int(threadIdx.x) >= quads) return;
  for (int j = 1; j < per; ++j) {
    const float4 v = acc_s[j * quads + threadIdx.x];
    acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
  }
  finish(span, mt.y, row, acc, top, sum);
}

StreamShape shape_of(int nb, int kt, int vt, int elem, int rows8) {
  switch (nb) {
    case 2: return paged::stream_shape<2>(kt, vt, elem, rows8);
    case 3: return paged::stream_shape<3>(kt, vt, elem, rows8);
    case 4: return paged::stream_shape<4>(kt, vt, elem, rows8);
    default: return paged::stream_shape<8>(kt, vt, elem, rows8);
  }
}

// A piece has at least this many tiles (of 16 or 32 tokens): below that a
// CTA's start and the combine cost more than the tokens (one sequence of 777
// tokens, 16 query over 8 kv heads of 128: 11.3 us with 2, 12.3 with 4, 13.3
// with 8).
constexpr int kMinTiles = 2;

// Sequences with more query rows per kv head than this go to the many-row
// kernel (16-bit calls, head_dim 64 or 128). A pass of the streaming kernel
// reads and converts the cache for 16 rows, a step of the other for 256, but
// the other's CTAs start slower and are fewer. Measured (8 kv heads of 128,
// 4 bits; streaming / many-row kernel): 16 sequences of 4096 tokens 69 / 70 us
// at 32 rows, 96 / 70 at 48, 122 / 70 at 64; one sequence of 8192 tokens 23.4 /
// 28.2 us at 48 rows, 26.2 / 28.4 at 64, 28.4 / 29.0 at 80, 39.6 / 30.0 at 128.
// So a batch that fills a quarter of the SMs by itself turns at 32, others at
// 64.
constexpr int kFill = 152;           // CTAs (one per SM) that the many-row kernel's split aims at
int tc_rows_of(int64_t n_seqs, int64_t n_kv) { return n_seqs * n_kv > kFill / 4 ? 32 : 64; }
// Tokens of a split at least (that one sequence at 64 rows: 256 tokens 29.9
// us, 512 28.4, 1024 31.5).
constexpr int kSplitTokens = 512;

struct Plan {
  StreamShape shape;
  int rows8, grid;
  int64_t items;  // many-row kernel: (kv head, 256 rows) pairs at most; 0: not launched
  int n_split;
  size_t part_o, part_ml, meta, tc_o, tc_ml, tc_meta, bytes;  // workspace offsets
};

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

Plan make_plan(PagedAttnArgs &a, int max_q, int sm_count) {
  Plan p = {};
  const int64_t most_rows = std::max<int64_t>(1, int64_t(a.group) * max_q), all_rows = int64_t(a.group) * a.n_q;
  const int tc_rows = tc_rows_of(a.n_seqs, a.sh.n_kv);
  const int64_t items = (all_rows / 256 + std::min<int64_t>(a.n_seqs, all_rows / (tc_rows + 1))) * a.sh.n_kv;
  const bool tc = a.elem != kElemF32 && (a.sh.nb == 2 || a.sh.nb == 4) && most_rows > tc_rows && items <= 0x7fffffff;
  a.tc_rows = tc ? tc_rows : 0x7fffffff;
  const int64_t rows = std::min<int64_t>(most_rows, a.tc_rows);
  p.rows8 = int(std::min<int64_t>((rows + 7) / 8, 1 << 20));
  p.shape = shape_of(a.sh.nb, a.kt, a.vt, a.elem, p.rows8);
  const int64_t seen = a.causal && a.window > 0 ? std::min<int64_t>(a.max_kv, int64_t(a.window) + max_q) : a.max_kv;
  const int64_t tiles = seen / p.shape.tokens + 2, groups = (rows + p.shape.rows - 1) / p.shape.rows;
  // saturating: only the smaller of this and the device's room matters
  const double most = double(tiles) * double(groups) * a.sh.n_kv * a.n_seqs / kMinTiles;
  const int room = std::min(sm_count, kMaxSms) * p.shape.ctas_per_sm;
  p.grid = most >= room ? room : std::max(1, int(most) + 1);
  p.n_split = 1;
  if (tc) {
    p.items = items;
    if (p.items > 0 && p.items <= kFill / 2)
      p.n_split = int(std::max<int64_t>(1, std::min<int64_t>(kFill / p.items, seen / kSplitTokens)));
  }
  const size_t D = size_t(a.sh.nb) * 32;
  auto take = [&](size_t &at, size_t n) {
    at = p.bytes;
    p.bytes += up256(n);
  };
  // the streaming part is sized for the largest device, whatever this one is
  const size_t srows = size_t(most >= kMaxSms * p.shape.ctas_per_sm ? kMaxSms * p.shape.ctas_per_sm : std::max(1, int(most) + 1)) * 2 * p.shape.rows;
  take(p.part_o, srows * D * 4);
  take(p.part_ml, srows * sizeof(float2));
  take(p.meta, size_t(kMaxCtas) * sizeof(int4));
  const size_t trows = p.n_split > 1 ? size_t(p.items) * size_t(p.n_split) * 256 : 0;
  take(p.tc_o, trows * D * 4);
  take(p.tc_ml, trows * sizeof(float2));
  take(p.tc_meta, trows ? size_t(p.items) * sizeof(int4) : 0);
  return p;
}

}  // namespace

bool paged_attn_dim(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 256; }

size_t paged_attn_workspace_bytes(PagedAttnArgs a, int max_q) { return make_plan(a, max_q, kMaxSms).bytes; }

cudaError_t launch_paged_attn(PagedAttnArgs a, int max_q, void *ws, cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  a.err = di->err_word;
  const Plan p = make_plan(a, max_q, di->sm_count);
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.part_o = reinterpret_cast<float *>(w + p.part_o);
  a.part_ml = reinterpret_cast<float2 *>(w + p.part_ml);
  a.meta = reinterpret_cast<int4 *>(w + p.meta);
  a.tc_part_o = reinterpret_cast<float *>(w + p.tc_o);
  a.tc_part_ml = reinterpret_cast<float2 *>(w + p.tc_ml);
  a.tc_meta = reinterpret_cast<int4 *>(w + p.tc_meta);
  const bool tc = p.items > 0;
  if (tc && (err = paged::launch_tc(a, p.items, p.n_split, stream)) != cudaSuccess) return err;
  switch (a.sh.nb) {
    case 2: err = paged::launch_stream<2>(a, p.rows8, p.grid, kMinTiles, tc, stream); break;
    case 3: err = paged::launch_stream<3>(a, p.rows8, p.grid, kMinTiles, tc, stream); break;
    case 4: err = paged::launch_stream<4>(a, p.rows8, p.grid, kMinTiles, tc, stream); break;
    default: err = paged::launch_stream<8>(a, p.rows8, p.grid, kMinTiles, tc, stream); break;
  }
  if (err != cudaSuccess) return err;
  const int D = a.sh.nb * 32, per = kCombineThreads / (D / 4);
  const int64_t tc_blocks = p.n_split > 1 ? p.items * ((256 + per - 1) / per) : 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.grid * p.shape.rows + tc_blocks));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_paged_combine, a, p.grid, p.shape.rows, D, p.n_split);
}

}  // namespace bq

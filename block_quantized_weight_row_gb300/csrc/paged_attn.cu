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

// Merges the partial results of one row of one split segment: block (i, r)
// takes the segment that starts in piece i, if there is one, and its row r.
// Bound by latency: at most a few megabytes of partials come out of L2. The
// weights 2^(m_i - max) are made once per partial, then 256 threads read the
// partials' rows as 16-byte vectors, D / 4 of them per row.
__global__ void __launch_bounds__(kCombineThreads) k_paged_combine(const __grid_constant__ PagedAttnArgs a, int rows, int D) {
  __shared__ float weight[kMaxCtas];
  __shared__ float red[kCombineThreads / 32][2];
  __shared__ float4 acc_s[kCombineThreads];
  pdl_wait();
  const int4 mt = a.meta[blockIdx.x];
  if (mt.w < 0) return;
  const SeqSpan span = paged::load_span(a, mt.x, false);
  const int row = mt.z * rows + int(blockIdx.y);
  if (row >= span.q_len * a.group) return;
  const int first = int(blockIdx.x), n = mt.w - first + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto part = [&](int i) { return (int64_t(first + i) * 2 + (i == 0 ? 1 : 0)) * rows + int64_t(blockIdx.y); };
  float top = -INFINITY;
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

  const int quads = D / 4, per = kCombineThreads / quads;  // `per` partials at a time
  const int ch = int(threadIdx.x) % quads * 4, k = int(threadIdx.x) / quads;
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
  const int tok = row / a.group, head = mt.y * a.group + (row - tok * a.group);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint8_t *out = a.o + int64_t(span.q0 + tok) * a.o_token + int64_t(head) * a.o_head;
  paged::store_out4(a.elem, out, ch, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (threadIdx.x == 0 && a.lse)
    a.lse[int64_t(span.q0 + tok) * a.n_heads + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / paged::kLog2e;
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
// CTA's start and the combine cost more than the tokens.
constexpr int kMinTiles = 4;

struct StreamPlan {
  StreamShape shape;
  int rows8, grid;
};

StreamPlan plan(const PagedAttnArgs &a, int max_q, int sm_count) {
  StreamPlan p;
  const int64_t rows = std::max<int64_t>(1, std::min<int64_t>(int64_t(a.group) * max_q, a.tc_rows));
  p.rows8 = int(std::min<int64_t>((rows + 7) / 8, 1 << 20));
  p.shape = shape_of(a.sh.nb, a.kt, a.vt, a.elem, p.rows8);
  const int64_t seen = a.causal && a.window > 0 ? std::min<int64_t>(a.max_kv, int64_t(a.window) + max_q) : a.max_kv;
  const int64_t tiles = seen / p.shape.tokens + 2, groups = (rows + p.shape.rows - 1) / p.shape.rows;
  // saturating: only the smaller of this and the device's room matters
  const double most = double(tiles) * double(groups) * a.sh.n_kv * a.n_seqs / kMinTiles;
  const int room = std::min(sm_count, kMaxSms) * p.shape.ctas_per_sm;
  p.grid = most >= room ? room : std::max(1, int(most) + 1);
  return p;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

bool paged_attn_dim(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 256; }

size_t paged_attn_workspace_bytes(const PagedAttnArgs &a, int max_q) {
  const StreamPlan p = plan(a, max_q, kMaxSms);
  const size_t rows = size_t(p.grid) * 2 * p.shape.rows;
  return up256(rows * a.sh.nb * 32 * 4) + up256(rows * sizeof(float2)) + up256(size_t(p.grid) * sizeof(int4));
}

cudaError_t launch_paged_attn(PagedAttnArgs a, int max_q, void *ws, cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  a.err = di->err_word;
  const StreamPlan p = plan(a, max_q, di->sm_count);
  const size_t rows = size_t(p.grid) * 2 * p.shape.rows;
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.part_o = reinterpret_cast<float *>(w);
  a.part_ml = reinterpret_cast<float2 *>(w + up256(rows * a.sh.nb * 32 * 4));
  a.meta = reinterpret_cast<int4 *>(w + up256(rows * a.sh.nb * 32 * 4) + up256(rows * sizeof(float2)));
  switch (a.sh.nb) {
    case 2: err = paged::launch_stream<2>(a, p.rows8, p.grid, kMinTiles, stream); break;
    case 3: err = paged::launch_stream<3>(a, p.rows8, p.grid, kMinTiles, stream); break;
    case 4: err = paged::launch_stream<4>(a, p.rows8, p.grid, kMinTiles, stream); break;
    default: err = paged::launch_stream<8>(a, p.rows8, p.grid, kMinTiles, stream); break;
  }
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.grid), unsigned(std::min(p.shape.rows, p.rows8 * 8)));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_paged_combine, a, p.shape.rows, a.sh.nb * 32);
}

}  // namespace bq

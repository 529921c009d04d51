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

// A load that stays where it is written (a plain one is moved down to its use)
__device__ __forceinline__ float4 load4_now(const float *p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

// Merges partial results. Of the first grid * rows / 8 blocks, block (i, g)
// takes rows 8 g .. 8 g + 7 of the split segment of the streaming kernel that
// starts in piece i, if there is one: a warp per row, or several where fewer
// rows are live, each with eight partial rows' loads in flight. The blocks
// after them take 1024 / D rows each of the many-row kernel's items. Bound by
// latency: at most a few megabytes come out of L2. A block of 256 threads per
// row starts in several waves (drafted tokens of 64 channels 27.7 us in all
// against 23.5, a decode batch 103.6 against 99.7); one warp per row leaves
// too few loads in flight (one sequence of 777 tokens 14.4 against 12.3). The
// order of the sums is fixed.
template <int NB>
__global__ void __launch_bounds__(kCombineThreads)
    k_paged_combine(const __grid_constant__ PagedAttnArgs a, int grid, int rows, int n_split) {
  constexpr int D = NB * 32, quads = D / 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  auto finish = [&](const SeqSpan &span, int kvh, int row, int ch, float4 acc, float top, float sum) {
    const int tok = row / a.group, head = kvh * a.group + (row - tok * a.group);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint8_t *out = a.o + int64_t(span.q0 + tok) * a.o_token + int64_t(head) * a.o_head;
    paged::store_out4(a.elem, out, ch, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (ch == 0 && a.lse)
      a.lse[int64_t(span.q0 + tok) * a.n_heads + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / paged::kLog2e;
  };
  auto add = [](float4 &acc, const float4 &v, float w) {
    acc.x = fmaf(v.x, w, acc.x), acc.y = fmaf(v.y, w, acc.y), acc.z = fmaf(v.z, w, acc.z), acc.w = fmaf(v.w, w, acc.w);
  };
  const int groups = rows / 8;
  if (int(blockIdx.x) >= grid * groups) {
    constexpr int per = kCombineThreads / quads;
    const int ch = int(threadIdx.x) % quads * 4, k = int(threadIdx.x) / quads;
    const int blocks = (256 + per - 1) / per, i = int(blockIdx.x) - grid * groups, item = i / blocks, r = (i - item * blocks) * per + k;
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
      sum = fmaf(ml.y, w, sum);
      add(acc, *reinterpret_cast<const float4 *>(a.tc_part_o + (p0 + s * 256) * D + ch), w);
    }
    finish(paged::load_span(a, mt.x, false), mt.y, mt.z + r, ch, acc, top, sum);
    return;
  }
  const int first = int(blockIdx.x) / groups, row8 = (int(blockIdx.x) - first * groups) * 8;
  const int4 mt = a.meta[first];
  if (mt.w < 0) return;
  const SeqSpan span = paged::load_span(a, mt.x, false);
  const int live = min(8, span.q_len * a.group - (mt.z * rows + row8));
  if (live <= 0) return;
  // W warps per row, the power of two that the live rows leave; a warp's
  // partials are W apart.
  const int lw = live > 4 ? 0 : live > 2 ? 1 : live > 1 ? 2 : 3, W = 1 << lw, sub = warp & (W - 1), r = row8 + (warp >> lw);
  const int pieces = mt.w - first + 1, n = r - row8 < live ? (pieces - sub + W - 1) >> lw : 0;
  auto part = [&](int t) {
    const int i = (t << lw) + sub;
    return (int64_t(first + i) * 2 + (i == 0 ? 1 : 0)) * rows + r;
  };
  // A lane holds Q quads of channels; with 64 channels the half-warps take
  // every second partial.
  constexpr int P = quads <= 16 ? 2 : 1, Q = (quads + 31) / 32, U = 8 / Q;
  const int half = P == 2 ? lane >> 4 : 0, ch = (P == 2 ? lane & 15 : lane) * 4;
  const float2 ml0 = lane < n ? a.part_ml[part(lane)] : make_float2(paged::kNoMax, 0.0f);
  float top = ml0.x;
  for (int i = lane + 32; i < n; i += 32) top = fmaxf(top, a.part_ml[part(i)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  float sum = 0.0f;
  float4 acc[Q] = {};
  for (int base = 0; base < n; base += 32) {
    const int mine = base + lane, m = min(32, n - base);
    float w = 0.0f;
    if (mine < n) {
      const float2 ml = base == 0 ? ml0 : a.part_ml[part(mine)];
      w = ml.y == 0.0f ? 0.0f : paged::ex2(ml.x - top);
      sum = fmaf(ml.y, w, sum);
    }
    for (int j = 0; j < m; j += P * U) {
      float4 v[U][Q];
      float wj[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = j + u * P + half;
        wj[u] = __shfl_sync(kFull, w, i & 31);
        if (i >= m) wj[u] = 0.0f;
        // no branch around the loads (at its end they would be waited for)
        const float *src = a.part_o + part(base + min(i, m - 1)) * D + (ch < D ? ch : 0);
#pragma unroll
        for (int q = 0; q < Q; ++q) v[u][q] = load4_now(src + 128 * q);
      }
      // where nothing was seen nothing was written
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < Q; ++q)
          if (wj[u] == 0.0f) v[u][q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < Q; ++q) add(acc[q], v[u][q], wj[u]);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if constexpr (P == 2) {
    acc[0].x += __shfl_xor_sync(kFull, acc[0].x, 16), acc[0].y += __shfl_xor_sync(kFull, acc[0].y, 16);
    acc[0].z += __shfl_xor_sync(kFull, acc[0].z, 16), acc[0].w += __shfl_xor_sync(kFull, acc[0].w, 16);
  }
  const bool holds = half == 0 && ch < D;
  if (W > 1) {  // the same for the whole block
    __shared__ float4 acc_s[8][quads];
    __shared__ float2 ml_s[8];
    if (holds)
#pragma unroll
      for (int q = 0; q < Q; ++q) acc_s[warp][ch / 4 + 32 * q] = acc[q];
    if (lane == 0) ml_s[warp] = make_float2(top, sum);
    __syncthreads();
    if (sub) return;
    for (int k = 1; k < W; ++k) top = fmaxf(top, ml_s[warp + k].x);
    sum = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < W; ++k) {
      const float2 ml = ml_s[warp + k];
      const float w = ml.y == 0.0f ? 0.0f : paged::ex2(ml.x - top);
      sum = fmaf(ml.y, w, sum);
      if (holds)
#pragma unroll
        for (int q = 0; q < Q; ++q) add(acc[q], acc_s[warp + k][ch / 4 + 32 * q], w);
    }
  }
  if (!holds || r - row8 >= live) return;
#pragma unroll
  for (int q = 0; q < Q; ++q) finish(span, mt.y, mt.z * rows + r, ch + 128 * q, acc[q], top, sum);
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
// tokens, 16 query over 8 kv heads of 128: 12.3 us with 2, 11.9 with 4, 13.3
// with 8).
constexpr int kMinTiles = 2;

// Sequences with more query rows per kv head than tc_rows_of go to the
// many-row kernel (16-bit calls, head_dim 64 or 128), if the call has work for
// it: kTcWork or more of passes x sequences x kv heads x (tokens + the 512 that
// a segment's start costs), by the host's bounds. A pass of the streaming
// kernel reads and converts the cache for 16 rows, a step of the other for
// 256, but the other's CTAs start slower (14 us an item) and are fewer.
// Measured (8 kv heads of 128, 4 bits; streaming / many-row kernel, us):
// sequences x tokens   rows 36    64         80         128        256        512
//  1 x 1024          11 / 20   15 / 21    16 / 21    17 / 22    21 / 27    31 / 29
//  1 x 8192                    26 / 24    28 / 24    40 / 25    66 / 40
//  4 x 256           15 / 16   16 / 15    17 / 16    21 / 16    32 / 19    49 / 20
// 16 x 512           31 / 20   38 / 20    45 / 21    62 / 20   111 / 23   214 / 43
// 16 x 4096 (48 rows 96 / 70) 122 / 71   149 / 71   227 / 71   440 / 85
// (16 x 4096 at 32 rows: 69 / 70.) All with 128 channels; the rule serves 64 as
// well. Work alone does not separate the entries: 4 x 256 at 128 rows and 1 x
// 1024 at 256 rows have the same, 196608, and with four times the items the
// first would be a quarter faster on the other kernel. A binary16 call turns at 64 rows at the
// earliest, as the many-row kernel's binary16 operands show in its output
// (4.5e-4 of its norm; streaming 2.9e-4, rounding alone 2.1e-4; a bf16
// output's rounding hides them: 1.7e-3 in all).
constexpr int kFill = 152;           // CTAs (one per SM) that the many-row kernel's split aims at
constexpr double kTcWork = 250000;
int tc_rows_of(int elem) { return elem == kElemBF16 ? 32 : 64; }
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
  const int64_t seen = a.causal && a.window > 0 ? std::min<int64_t>(a.max_kv, int64_t(a.window) + max_q) : a.max_kv;
  const int tc_rows = tc_rows_of(a.elem);
  const bool work = double((most_rows + 15) / 16) * double(a.n_seqs) * a.sh.n_kv * double(seen + 512) >= kTcWork;
  const int64_t items = (all_rows / 256 + std::min<int64_t>(a.n_seqs, all_rows / (tc_rows + 1))) * a.sh.n_kv;
  const bool tc = a.elem != kElemF32 && (a.sh.nb == 2 || a.sh.nb == 4) && work && most_rows > tc_rows && items <= 0x7fffffff;
  a.tc_rows = tc ? tc_rows : 0x7fffffff;
  const int64_t rows = std::min<int64_t>(most_rows, a.tc_rows);
  p.rows8 = int(std::min<int64_t>((rows + 7) / 8, 1 << 20));
  p.shape = shape_of(a.sh.nb, a.kt, a.vt, a.elem, p.rows8);
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

int64_t paged_attn_many_rows(PagedAttnArgs a, int max_q) { return make_plan(a, max_q, kMaxSms).items > 0 ? a.tc_rows : 0; }

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
  cfg.gridDim = dim3(unsigned(p.grid * (p.shape.rows / 8) + tc_blocks));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (a.sh.nb) {
    case 2: return cudaLaunchKernelEx(&cfg, k_paged_combine<2>, a, p.grid, p.shape.rows, p.n_split);
    case 3: return cudaLaunchKernelEx(&cfg, k_paged_combine<3>, a, p.grid, p.shape.rows, p.n_split);
    case 4: return cudaLaunchKernelEx(&cfg, k_paged_combine<4>, a, p.grid, p.shape.rows, p.n_split);
    default: return cudaLaunchKernelEx(&cfg, k_paged_combine<8>, a, p.grid, p.shape.rows, p.n_split);
  }
}

}  // namespace bq

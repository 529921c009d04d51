// paged_extend.cu — page tables, slots and positions of a batch's next tokens,
// made on the GPU from the sequences' lengths (include/bq.h: bq_paged_extend).
//
// With owned_b = ceil(kv_b / P) and need_b = ceil((kv_b + n_b) / P) - owned_b,
// sequence b takes free pages base_b .. base_b + need_b - 1 (base: the sum of
// the needs before it) and its tokens the rows start_b .. (start: the sum of
// the n before it). Two prefix sums over the sequences, then one page and one
// slot per token.
//
// Bound by latency (a decode step) or by the 12 bytes written per token. One
// launch without a workspace: every CTA sums up all sequences itself (8 bytes
// each, from L2 after the first CTA; 0.2 us for 8192), which costs less than a
// second launch or a wait among CTAs, and then makes its own tiles of tokens.
// A tile's tokens find their sequence by a running maximum over the tile: each
// sequence puts its record at its first token in the tile.
#include <algorithm>
#include <climits>

#include "bq_device.cuh"
#include "bq_internal.h"
#include "layer.h"

namespace bq {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 2;  // tokens of a thread: one 16-byte store of slots
constexpr int kTile = kThreads * kPerThread;
constexpr uint32_t kCap = 0x7fffffffu;

// Sums saturate at 2^31 - 1, above every count that can be met: saturating
// addition is associative, so the prefix sums may be cut anywhere.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kCap); }

struct Seq {
  uint32_t kv, n, need;
  bool ok;  // lengths that are none, or longer than the table, get nothing
};

__device__ __forceinline__ Seq load_seq(const ExtendArgs &a, int b) {
  const int kv = __ldg(a.kv_len + b), n = __ldg(a.n_new + b);
  Seq s;
  s.kv = uint32_t(max(kv, 0));
  s.n = uint32_t(max(n, 0));
  const uint32_t end = s.kv + s.n;  // below 2^32
  s.ok = kv >= 0 && n >= 0 && end <= a.max_tokens;
  const uint32_t P = a.page_size;
  s.need = s.ok ? (end + P - 1) / P - (s.kv + P - 1) / P : 0;
  return s;
}

struct Record {
  uint32_t kv, start;  // cached tokens; the batch's row of the first new one
  int seq, base;       // base: place in the free list of page column 0, if that were new; INT_MIN: the sequence gets nothing
};

__global__ void __launch_bounds__(kThreads) k_paged_extend(const ExtendArgs a) {
  __shared__ Record rec[kTile];
  __shared__ int head[kTile];  // the token itself where a sequence begins in the tile, else -1
  __shared__ uint32_t sums[2][kWarps];
  __shared__ int warp_head[kWarps];
  __shared__ uint32_t most;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.n_seqs, chunk = (B + kThreads - 1) / kThreads;
  const int b0 = min(tid * chunk, B), b1 = min(b0 + chunk, B);
  if (tid == 0) most = 0;

  // ---- this thread's sequences, then the sums before them ----
  uint32_t tokens = 0, pages = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    const Seq s = load_seq(a, b);
    tokens = sat_add(tokens, s.n);
    pages = sat_add(pages, s.need);
  }
  uint32_t ti = tokens, pi = pages;  // inclusive over the warp
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t t = __shfl_up_sync(kFull, ti, d), p = __shfl_up_sync(kFull, pi, d);
    if (lane >= d) ti = sat_add(ti, t), pi = sat_add(pi, p);
  }
  if (lane == 31) sums[0][warp] = ti, sums[1][warp] = pi;
  uint32_t t0 = __shfl_up_sync(kFull, ti, 1), p0 = __shfl_up_sync(kFull, pi, 1);
  if (lane == 0) t0 = p0 = 0;
  __syncthreads();
  uint32_t all_tokens = 0, all_pages = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) t0 = sat_add(t0, all_tokens), p0 = sat_add(p0, all_pages);
    all_tokens = sat_add(all_tokens, sums[0][w]);
    all_pages = sat_add(all_pages, sums[1][w]);
  }
  const uint32_t t_end = sat_add(t0, tokens);

  // ---- the per-sequence outputs of this CTA's share, and its tiles ----
  const int s0 = int(int64_t(B) * blockIdx.x / gridDim.x), s1 = int(int64_t(B) * (blockIdx.x + 1) / gridDim.x);
  const uint32_t n_slots = a.n_slots, P = a.page_size;
  unsigned bad = 0;
  bool first = true;
  for (uint32_t tile = blockIdx.x;; tile += gridDim.x) {
    const uint64_t lo = uint64_t(tile) * kTile;
    const bool live = lo < n_slots;
    if (!live && !first) break;
    const uint32_t hi = uint32_t(min(lo + kTile, uint64_t(n_slots)));
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) head[tid + i * kThreads] = -1;
    __syncthreads();
    const bool mine = first && b0 < s1 && b1 > s0;              // some outputs of this thread's sequences are this CTA's
    const bool meets = live && t0 < hi && t_end > uint32_t(lo);  // some of its tokens are in the tile
    if (mine || meets || (first && blockIdx.x == 0)) {
      uint32_t start = t0, base = p0;
#pragma unroll 4
      for (int b = b0; b < b1; ++b) {
        const Seq s = load_seq(a, b);
        const uint32_t end = sat_add(start, s.n);
        const bool gets = s.ok && (s.n == 0 || (end <= n_slots && end < kCap)) && (s.need == 0 || sat_add(base, s.need) <= a.n_free);
        if (first && b >= s0 && b < s1) {
          a.q_start[b + 1] = int(end);
          a.kv_out[b] = gets ? int(s.kv + s.n) : a.kv_len[b];
          if (!gets) bad = kErrIndex;
        }
        if (first && blockIdx.x == 0 && gets && s.need) atomicMax(&most, base + s.need);
        if (live && s.n && start < hi && end > uint32_t(lo)) {
          const uint32_t at = max(start, uint32_t(lo)) - uint32_t(lo);
          const uint32_t owned = (s.kv + P - 1) / P;
          rec[at] = Record{s.kv, start, b, gets ? int(base) - int(owned) : INT_MIN};
          head[at] = int(at);
        }
        start = end;
        base = sat_add(base, s.need);
      }
    }
    __syncthreads();
    if (first && blockIdx.x == 0 && tid == 0) {
      a.q_start[0] = 0;
      a.taken[0] = int(most);
      a.taken[1] = int(all_pages);
    }
    first = false;
    if (!live) break;

    // ---- the latest sequence that began at or before each token ----
    const int at = tid * kPerThread;
    int h[kPerThread], m = -1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) h[i] = m = max(m, head[at + i]);
    int run = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, run, d);
      if (lane >= d) run = max(run, o);
    }
    if (lane == 31) warp_head[warp] = run;
    int before = __shfl_up_sync(kFull, run, 1);
    if (lane == 0) before = -1;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before = max(before, warp_head[w]);

    longlong2 slot;
    int pos[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const uint64_t t = lo + at + i;
      const int k = max(h[i], before);
      int64_t sl = -1;
      pos[i] = 0;
      if (t < n_slots && t < all_tokens && k >= 0) {
        const Record r = rec[k];
        const uint32_t p = r.kv + (uint32_t(t) - r.start);
        pos[i] = int(min(p, kCap));
        if (r.base != INT_MIN) {
          const uint32_t col = p / P, place = p - col * P;
          int32_t *entry = a.page_table + int64_t(r.seq) * a.max_pages + col;
          const bool fresh = col >= (r.kv + P - 1) / P;
          const int page = fresh ? __ldg(a.free_pages + (r.base + int(col))) : *entry;
          if (uint32_t(page) < a.n_pages) {
            if (fresh && (place == 0)) *entry = page;
            sl = int64_t(page) * P + place;
          } else {
            bad = kErrIndex;
          }
        }
      }
      (i == 0 ? slot.x : slot.y) = sl;
    }
    const uint64_t t = lo + at;
    if (t + 1 < n_slots && a.wide) {
      *reinterpret_cast<longlong2 *>(a.slots + t) = slot;
      if (a.positions) *reinterpret_cast<int2 *>(a.positions + t) = make_int2(pos[0], pos[1]);
    } else {
      if (t < n_slots) {
        a.slots[t] = slot.x;
        if (a.positions) a.positions[t] = pos[0];
      }
      if (t + 1 < n_slots) {
        a.slots[t + 1] = slot.y;
        if (a.positions) a.positions[t + 1] = pos[1];
      }
    }
    __syncthreads();  // the next tile writes rec and head
  }
  if (bad) atomicOr(a.err, bad);
}

}  // namespace

cudaError_t launch_paged_extend(ExtendArgs a, cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  a.err = di->err_word;
  a.wide = reinterpret_cast<uintptr_t>(a.slots) % 16 == 0 && reinterpret_cast<uintptr_t>(a.positions) % 8 == 0;
  const int64_t tiles = (int64_t(a.n_slots) + kTile - 1) / kTile;
  const int64_t shares = (int64_t(a.n_seqs) + 8 * kThreads - 1) / (8 * kThreads);
  const int64_t grid = std::min<int64_t>(std::max<int64_t>(std::max(tiles, shares), 1), int64_t(di->sm_count) * 4);
  k_paged_extend<<<unsigned(grid), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace bq

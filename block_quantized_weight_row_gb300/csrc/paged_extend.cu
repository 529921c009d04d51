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
// each, from L2 after the first CTA), which costs less than a second launch or a
// wait among CTAs, keeps the sums of chunks of 32 sequences, and then makes its
// own tiles of tokens: a warp per chunk that reaches into the tile puts each
// sequence's record at its first token there, and the tokens find theirs by a
// running maximum over the tile. 64 sequences of one token 4 us, 300 sequences of
// 200000 tokens 7 us, 8192 sequences of 936000 tokens 16 us.
#include <algorithm>
#include <climits>

#include "bq_device.cuh"
#include "bq_internal.h"
#include "layer.h"

namespace bq {
namespace {

constexpr int kMaxChunks = 1024;  // chunks of 32 sequences, or of several times 32 beyond 32768 sequences
constexpr uint32_t kCap = 0x7fffffffu;

// Sums saturate at 2^31 - 1, above every count that can be met: saturating
// addition is associative, so the prefix sums may be cut anywhere.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kCap); }

__device__ __forceinline__ uint32_t sat_sum_warp(uint32_t v) {  // v up to kCap: halves of 16 bits, whose sums fit
  const uint64_t hi = __reduce_add_sync(kFull, v >> 16), lo = __reduce_add_sync(kFull, v & 0xffffu);
  return uint32_t(min((hi << 16) + lo, uint64_t(kCap)));
}
__device__ __forceinline__ uint32_t sat_scan_warp(uint32_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(kFull, v, d);
    if (lane >= d) v = sat_add(v, o);
  }
  return v;
}

// x / page_size: x / 16 is below 2^28 and page_size / 16 up to 2^16, so the
// product with the rounded-up reciprocal errs by less than 2^44 / 2^64
__device__ __forceinline__ uint32_t pages_of(const ExtendArgs &a, uint32_t x) {
  return a.page_shift >= 0 ? x >> a.page_shift : uint32_t(__umul64hi(uint64_t(x >> 4), a.page_magic));
}

struct Seq {
  uint32_t kv, n, owned, need;
  bool ok;  // lengths that are none, or longer than the table, get nothing
};

__device__ __forceinline__ Seq load_seq(const ExtendArgs &a, int b) {
  Seq s{0, 0, 0, 0, true};
  if (b >= a.n_seqs) return s;
  const int kv = __ldg(a.kv_len + b), n = __ldg(a.n_new + b);
  s.kv = uint32_t(max(kv, 0));
  s.n = uint32_t(max(n, 0));
  const uint32_t end = s.kv + s.n;  // below 2^32
  s.ok = kv >= 0 && n >= 0 && end <= a.max_tokens;
  s.owned = pages_of(a, s.kv + a.page_size - 1);
  s.need = s.ok ? pages_of(a, end + a.page_size - 1) - s.owned : 0;
  return s;
}

struct Record {
  uint32_t kv, start;  // cached tokens; the batch's row of the first new one
  int seq, base;       // base: place in the free list of page column 0, if that were new; INT_MIN: the sequence gets nothing
};

// NT threads with kPerThread tokens of a tile each; chunks of 32 * rounds sequences
template <int NT, int kPerThread>
__global__ void __launch_bounds__(NT, 1) k_paged_extend(const ExtendArgs a, const int chunks, const int rounds) {
  constexpr int kWarps = NT / 32, kTile = NT * kPerThread, kEach = kMaxChunks / NT;
  extern __shared__ __align__(16) Record rec[];           // of the sequence that begins at a token of the tile
  __shared__ __align__(8) short head[kTile];  // the token itself where a sequence begins in the tile, else -1
  __shared__ uint32_t tok[kMaxChunks + 1], pag[kMaxChunks + 1];  // sums of a chunk, then before it
  __shared__ uint32_t sums[2][kWarps];
  __shared__ int warp_head[kWarps];
  __shared__ short met[kMaxChunks];
  __shared__ int n_met;
  __shared__ uint32_t most;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t n_slots = a.n_slots, P = a.page_size;
  if (tid == 0) most = 0;

  // ---- the sums of all chunks, then those before each ----
  constexpr int kAhead = 4;  // chunks of a warp whose lengths are in flight
  for (int c0 = warp; c0 < chunks; c0 += kAhead * kWarps) {
    uint32_t t[kAhead] = {}, p[kAhead] = {};
    for (int r = 0; r < rounds; ++r) {
      Seq s[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) s[k] = c0 + k * kWarps < chunks ? load_seq(a, ((c0 + k * kWarps) * rounds + r) * 32 + lane) : Seq{0, 0, 0, 0, true};
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        t[k] = sat_add(t[k], s[k].n);
        p[k] = sat_add(p[k], s[k].need);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int c = c0 + k * kWarps;
      if (c < chunks) {  // the warp's
        t[k] = sat_sum_warp(t[k]);
        p[k] = sat_sum_warp(p[k]);
        if (lane == 0) tok[c] = t[k], pag[c] = p[k];
      }
    }
  }
  __syncthreads();
  uint32_t t = 0, p = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (tid * kEach + i < chunks) t = sat_add(t, tok[tid * kEach + i]), p = sat_add(p, pag[tid * kEach + i]);
  const uint32_t ti = sat_scan_warp(t, lane), pi = sat_scan_warp(p, lane);
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
#pragma unroll
  for (int i = 0; i < kEach; ++i) {  // each thread its own entries
    const int c = tid * kEach + i;
    if (c < chunks) {
      const uint32_t x = tok[c], y = pag[c];
      tok[c] = t0, pag[c] = p0;
      t0 = sat_add(t0, x), p0 = sat_add(p0, y);
    }
  }
  if (tid == 0) tok[chunks] = all_tokens;
  __syncthreads();

  unsigned bad = 0;
  // A chunk by a warp: f(sequence's index, sequence, start, end, base, whether it grows).
  auto each = [&](int c, auto f) {
    uint32_t start = tok[c], base = pag[c];
    for (int r = 0; r < rounds; ++r) {
      const int b = (c * rounds + r) * 32 + lane;
      const Seq s = load_seq(a, b);
      const uint32_t ends = sat_scan_warp(s.n, lane), needs = sat_scan_warp(s.need, lane);
      uint32_t before = __shfl_up_sync(kFull, ends, 1), pages = __shfl_up_sync(kFull, needs, 1);
      if (lane == 0) before = pages = 0;
      const uint32_t from = sat_add(start, before), to = sat_add(start, ends), first = sat_add(base, pages);
      const bool gets = s.ok && (s.n == 0 || (to <= n_slots && to < kCap)) && (s.need == 0 || sat_add(first, s.need) <= a.n_free);
      if (b < a.n_seqs) f(b, s, from, to, first, gets);
      start = sat_add(start, __shfl_sync(kFull, ends, 31));
      base = sat_add(base, __shfl_sync(kFull, needs, 31));
    }
  };

  // ---- outputs per sequence: the chunks shared out over the grid ----
  for (int c = blockIdx.x + warp * gridDim.x; c < chunks; c += kWarps * gridDim.x)
    each(c, [&](int b, const Seq &s, uint32_t, uint32_t to, uint32_t, bool gets) {
      a.q_start[b + 1] = int(to);
      a.kv_out[b] = gets ? int(s.kv + s.n) : a.kv_len[b];
      if (!gets) bad = kErrIndex;
    });
  if (blockIdx.x == 0) {
    // where pages and slots suffice, every sequence that needs pages gets them
    const bool enough = all_pages <= a.n_free && all_tokens <= n_slots && all_tokens < kCap;
    if (!enough) {
      for (int c = warp; c < chunks; c += kWarps)
        each(c, [&](int, const Seq &s, uint32_t, uint32_t, uint32_t first, bool gets) {
          if (gets && s.need) atomicMax(&most, first + s.need);
        });
      __syncthreads();
    }
    if (tid == 0) {
      a.q_start[0] = 0;
      a.taken[0] = int(enough ? all_pages : most);
      a.taken[1] = int(all_pages);
    }
  }

  for (uint64_t lo64 = uint64_t(blockIdx.x) * kTile; lo64 < n_slots; lo64 += uint64_t(gridDim.x) * kTile) {
    const uint32_t lo = uint32_t(lo64), hi = uint32_t(min(lo64 + kTile, uint64_t(n_slots)));
    // ---- records of the sequences with tokens in the tile ----
    if (tid == 0) n_met = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) head[tid + i * NT] = -1;
    __syncthreads();
    for (int c = tid; c < chunks; c += NT)
      if (tok[c] < hi && tok[c + 1] > lo) met[atomicAdd(&n_met, 1)] = short(c);
    __syncthreads();
    for (int k = warp; k < n_met; k += kWarps)
      each(met[k], [&](int b, const Seq &s, uint32_t from, uint32_t to, uint32_t first, bool gets) {
        if (s.n && from < hi && to > lo) {
          const uint32_t i = max(from, lo) - lo;
          rec[i] = Record{s.kv, from, b, gets ? int(first) - int(s.owned) : INT_MIN};
          head[i] = short(i);
        }
      });
    __syncthreads();

    // ---- the latest sequence that began at or before each token ----
    const int at = tid * kPerThread;
    int h[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) h[i] = i ? max(int(head[at + i]), h[i ? i - 1 : 0]) : head[at];
    int run = h[kPerThread - 1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, run, d);
      if (lane >= d) run = max(run, o);
    }
    if (lane == 31) warp_head[warp] = run;
    int before = __shfl_up_sync(kFull, run, 1);
    if (lane == 0) before = -1;
    __syncthreads();
    before = max(before, __reduce_max_sync(kFull, lane < warp ? warp_head[lane] : -1));

    long long slot[kPerThread];
    int pos[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const uint32_t t = lo + at + i;
      const int k = max(h[i], before);
      slot[i] = -1;
      pos[i] = 0;
      if (t < n_slots && t < all_tokens && k >= 0) {
        const Record r = rec[k];
        const uint32_t p = r.kv + (t - r.start);
        pos[i] = int(min(p, kCap));
        if (r.base != INT_MIN) {
          const uint32_t col = pages_of(a, p), place = p - col * P;
          int32_t *entry = a.page_table + int64_t(r.seq) * a.max_pages + col;
          const bool fresh = col >= pages_of(a, r.kv + P - 1);
          const int page = fresh ? __ldg(a.free_pages + (r.base + int(col))) : *entry;
          if (uint32_t(page) < a.n_pages) {
            if (fresh && place == 0) *entry = page;
            slot[i] = int64_t(page) * P + place;
          } else {
            bad = kErrIndex;
          }
        }
      }
    }
    const uint32_t t = lo + at;
    if (t + kPerThread <= n_slots && a.wide) {
#pragma unroll
      for (int i = 0; i < kPerThread; i += 2) {
        *reinterpret_cast<longlong2 *>(a.slots + t + i) = make_longlong2(slot[i], slot[i + 1]);
        if (a.positions) *reinterpret_cast<int2 *>(a.positions + t + i) = make_int2(pos[i], pos[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i)
        if (t + i < n_slots) {
          a.slots[t + i] = slot[i];
          if (a.positions) a.positions[t + i] = pos[i];
        }
    }
    __syncthreads();  // the next tile writes rec, head and met
  }
  if (bad) atomicOr(a.err, bad);
}

template <int NT, int PT>
cudaError_t launch(const ExtendArgs &a, int sms, cudaStream_t stream) {
  const int rounds = std::max(1, (a.n_seqs + 32 * kMaxChunks - 1) / (32 * kMaxChunks));
  const int chunks = (a.n_seqs + 32 * rounds - 1) / (32 * rounds);
  constexpr int kTile = NT * PT, kSmem = kTile * int(sizeof(Record));
  const int64_t tiles = (int64_t(a.n_slots) + kTile - 1) / kTile, shares = (chunks + NT / 32 - 1) / (NT / 32);
  // one CTA per SM at most: each sums up all sequences
  const int64_t grid = std::min<int64_t>(std::max<int64_t>(std::max(tiles, shares), 1), sms);
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(k_paged_extend<NT, PT>), kSmem);
  if (e != cudaSuccess) return e;
  k_paged_extend<NT, PT><<<unsigned(grid), NT, kSmem, stream>>>(a, chunks, rounds);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_extend(ExtendArgs a, cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  a.err = di->err_word;
  a.wide = reinterpret_cast<uintptr_t>(a.slots) % 16 == 0 && reinterpret_cast<uintptr_t>(a.positions) % 8 == 0;
  a.page_shift = -1;
  for (int k = 4; k <= 20; ++k)
    if (a.page_size == 1u << k) a.page_shift = k;
  a.page_magic = ~uint64_t(0) / (a.page_size / 16) + 1;
  // a decode step of a few hundred sequences: fewer threads meet at a barrier sooner
  if (a.n_seqs <= 512 && a.n_slots <= 2048) return launch<256, 2>(a, di->sm_count, stream);
  // small tiles as long as every SM has one at most; then fewer turns count (936000 tokens: 15.3 us for 18.4)
  if (int64_t(a.n_slots) <= int64_t(di->sm_count) * 2048) return launch<1024, 2>(a, di->sm_count, stream);
  return launch<1024, 4>(a, di->sm_count, stream);
}

}  // namespace bq

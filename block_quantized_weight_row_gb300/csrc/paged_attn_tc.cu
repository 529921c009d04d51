// paged_attn_tc.cu — attention of many query rows per kv head over a paged,
// block-quantized KV cache (prompt chunks) on the fifth-generation tensor
// cores: the many-row kernel, for bf16 and binary16 calls with 64 or 128
// channels.
//
// Bound by the tensor pipe and the issue slots together: 4 D flops per (row,
// token), one exponential and ~3 further operations beside them; converting
// the cache's codes is shared by the 256 rows of a CTA. Measured, a chunk of
// 2048 tokens at 8192, 32 query over 8 kv heads of 128, 4 bits: 268 us, 898
// TFLOP/s (0.47 of the measured bf16 rate). A step takes 4300 cycles; its
// products alone, issued without a wait, 2520 (2048 where S is 128 tokens wide:
// 64 tokens' operands are fetched at 49 cycles per product, not 33), its 11600
// instructions 2900 issue slots of each scheduler. 11 us of an item are its
// start and its output, and 256 items on 152 SMs leave a sixth of them idle in
// the second wave. A step is 256 rows x 128 tokens:
//   - S = Q K^T per 128-row tile and 64 tokens (operands in shared memory,
//     accumulator in tensor memory), softmax by one thread per row, P back
//     into tensor memory over S as binary16, O += P V with P as the
//     tensor-memory operand. Two row tiles and two halves of the tokens are in
//     flight: while a warp works on one half, the tensor pipe finishes P V and
//     the next S of the other (one 128-token S per row tile leaves each softmax
//     warp waiting for its own products: 330 us a chunk).
//   - A thread reads its row of S once: weights are made with the maximum as it
//     was and kept in registers; only if a score passed it by 2^8 are they made
//     again, with the row read again, before they are written over S.
//   - K and V operands are made from the page bytes on the way into shared
//     memory: k^ = d c as binary16, tokens x channels; V transposed, channels
//     x tokens, so that both are plain K-major operands (128-byte swizzle).
//     Channel orders inside the operands are those in which the code words
//     fall apart (Q and the output rows use the same permutation). Rounding d
//     c, q and the weights to binary16 costs 2^-11 each, an eighth of a bf16
//     output's own rounding; scales enter relative to the largest of 32
//     tokens (brought to [2^5, 2^6) by a power of two, undone in fp32), so that
//     neither large nor tiny scales leave binary16's range.
//   - Maxima are raised only when passed by 2^8; weights are 2^(s - m + 6).
// Warps: 0-3 and 4-7 softmax of row tiles A and B (and Q before, O after),
// 8-11 K operand, 12-15 V operand, 16 and 17 MMA issue for A and B, 18 and 19
// none (they complete a warpgroup whose registers go to the softmax). Waits are
// bounded as in the GEMM: one that runs out sets the error word, every role
// leaves, MMAs in flight are waited for and the tensor memory is freed.
// With few CTAs the tokens of a row tile are split over several, whose
// partial results the combine merges.
#include <cfloat>

#include "paged_attn.cuh"
#include "tcgen05.cuh"

namespace bq {
namespace paged {
namespace {

constexpr int kTcWarps = 20;
constexpr int kTcThreads = kTcWarps * 32;
constexpr int kTile = 128;  // tokens per step, rows per row tile
constexpr int kHead = 6;    // weights carry 2^kHead
constexpr int kSub = 128 * 128;  // bytes of an operand sub-tile: 128 rows x 64 binary16

// kSFull, kPReady: [row tile][half]. A phase of a barrier counts each of its
// arrivals once: no thread may arrive for a later phase while the one before is
// open. The empty barriers see to it for all but one, the V warps' arrival
// on kKFull (their exponents), which comes before their wait for kVEmpty: it
// waits for the phase of two tiles before itself.
enum Bar { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPReady = 12, kODone = 16, kAllDone = 18, kQReady = 20, kBars = 21 };

struct Misc {
  uint32_t tmem;
  int abort_flag;
  int kx[4][4], vx[4][4];  // [tile & 3][32 tokens]: their operand holds d c 2^x
  int64_t find[2];
  int64_t scan[kTcWarps];
};

template <int NB>
struct TcCfg {
  static constexpr int D = NB * 32, kSubs = D / 64;
  static constexpr int kQBytes = kSubs * kSub;                // one row tile
  static constexpr int kKBytes = kSubs * kSub;                // one K stage
  static constexpr int kVSub = D * 128, kVBytes = 2 * kVSub;  // one V stage: two halves of 64 tokens
  static constexpr int kOffK = 2 * kQBytes, kOffV = kOffK + 2 * kKBytes, kOffBar = kOffV + 2 * kVBytes;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kSmem = kOffMisc + int(sizeof(Misc)) + 1024;  // + slack to align the base to 1024
};

// D (tensor memory) (+)= A (tensor memory) * B (shared memory)
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Bounded wait that gives up once another thread has: a test, then waits that
// suspend the thread in the barrier unit. (Polling between naps, as the GEMM
// does, took a third of this kernel's issue slots.)
__device__ __forceinline__ bool pa_wait(uint64_t *bar, uint32_t parity, uint32_t limit, volatile int *abort_flag, unsigned *err) {
  for (uint32_t i = 0; i < limit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 15) == 15 && *abort_flag) return false;
  }
  *abort_flag = 1;
  atomicOr(err, kErrTimeout);
  return false;
}
// The same for a whole warp, every lane waiting for itself.
__device__ __forceinline__ bool pa_wait_warp(uint64_t *bar, uint32_t parity, uint32_t limit, volatile int *abort_flag, unsigned *err) {
  const bool ok = pa_wait(bar, parity, limit, abort_flag, err);
  return __all_sync(kFull, ok);
}

// H64 x / 8 of 64 values of one thread, spans 1 .. 32 in order
__device__ __forceinline__ void hadamard64_thread(float (&x)[64]) {
#pragma unroll
  for (int span = 1; span < 64; span <<= 1)
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if ((i & span) == 0) {
        const float a = x[i], b = x[i + span];
        x[i] = __fadd_rn(a, b);
        x[i + span] = __fsub_rn(a, b);
      }
#pragma unroll
  for (int i = 0; i < 64; ++i) x[i] *= 0.125f;
}

// Row r's 64 q values at its swizzled place in an operand sub-tile, as they
// were copied there
__device__ __forceinline__ void load_q64(int elem, const uint8_t *sub, int r, int rotate, float (&x)[64]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 v = *reinterpret_cast<const uint4 *>(sub + sw128_off(r, i));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = elem == kElemF16 ? unpack_pair<kElemF16>(w[k]) : unpack_pair<kElemBF16>(w[k]);
      x[8 * i + 2 * k] = f.x;
      x[8 * i + 2 * k + 1] = f.y;
    }
  }
  if (rotate) hadamard64_thread(x);
}

// Global loads that stay where they are written: a plain load may be moved
// down to its first use, which here is a tile later, behind the waits.
__device__ __forceinline__ int ldg_now(const int32_t *p) {
  int v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
// N bytes (a multiple of 4)
template <int N>
__device__ __forceinline__ void ldg_piece(const uint8_t *p, uint32_t (&w)[N / 4]) {
  if constexpr (N % 16 == 0) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i)
      asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "l"(p + 16 * i));
  } else if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(w[2 * i]), "=r"(w[2 * i + 1]) : "l"(p + 8 * i));
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(w[i]) : "l"(p + 4 * i));
  }
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Exponent k of the power of two that brings the largest of a warp's scales
// (pairs of binary16, not negative) to [2^5, 2^6); at most 2^15, which
// binary16 holds (scales below 2^-10 then stay below 2^5, all the same exact).
__device__ __forceinline__ int scale_up(uint32_t m) {
  const uint32_t e = __reduce_max_sync(kFull, max(m & 0x7fffu, (m >> 16) & 0x7fffu)) >> 10;
  return min(20 - int(e), 15);
}
// 2^k twice, -14 <= k <= 15
__device__ __forceinline__ uint32_t half2_pow2(int k) { return uint32_t(15 + k) * 0x04000400u; }

__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }

// Registers per thread: 96 at launch (20 warps); the shares add up to 20 * 96
// or less: 8 * 136 + 8 * 72 + 4 * 56 = 1888 or 8 * 136 + 8 * 80 + 4 * 48 =
// 1920 of 1920. Each is the split that leaves nothing in local memory (8 bytes
// with 8-bit K and 4-bit V); 128 / 88 / 40 took 284 us where 136 / 72 / 56
// takes 270.
template <int VT>
struct Regs {
  static constexpr bool kV4 = VT == kTypeQ4_0;
  static constexpr int kSoftmax = 136, kOperand = kV4 ? 72 : 80, kIssue = kV4 ? 56 : 48;
};
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int NB, int KT, int VT>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_paged_tc(const __grid_constant__ PagedAttnArgs a, int n_split, uint32_t spin) {
  using C = TcCfg<NB>;
  constexpr int D = C::D;
  constexpr bool K4 = KT == kTypeQ4_0, V4 = VT == kTypeQ4_0;
  constexpr int RBK = NB * Codes<KT>::kBytes, RBV = NB * Codes<VT>::kBytes;
  constexpr int UK = RBK / kUnitsK, UV = RBV / kUnitsV;
  constexpr uint32_t kIdescS = (1u << 4) | (uint32_t(64 >> 3) << 17) | (uint32_t(128 >> 4) << 24);
  constexpr uint32_t kIdescO = (1u << 4) | (uint32_t(D >> 3) << 17) | (uint32_t(128 >> 4) << 24);
  extern __shared__ uint8_t smem_dyn[];
  const uint32_t base = smem_u32(smem_dyn);
  uint8_t *sm = smem_dyn + (((base + 1023u) & ~1023u) - base);
  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
  Misc *mi = reinterpret_cast<Misc *>(sm + C::kOffMisc);
  volatile int *abort_flag = &mi->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();  // the streaming kernel of the same call shares no output with this one

  // ---- this CTA's item: sequence, kv head, 256 rows, share of the tokens ----
  const int64_t item = blockIdx.x / n_split;
  const int split = int(blockIdx.x - item * n_split);
  const int per_thread = (a.n_seqs + kTcThreads - 1) / kTcThreads;
  const int b_first = min(int(threadIdx.x) * per_thread, a.n_seqs), b_last = min(b_first + per_thread, a.n_seqs);
  auto row_tiles = [&](const SeqSpan &s) {
    const int n = s.q_len * a.group;
    return n > a.tc_rows ? int64_t((n + 255) / 256) * a.sh.n_kv : int64_t(0);
  };
  int64_t mine = 0;
  for (int b = b_first; b < b_last; ++b) mine += row_tiles(load_span(a, b, false));
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) mi->scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < kTcWarps; ++w) {
    if (w < warp) before += mi->scan[w];
    total += mi->scan[w];
  }
  if (item >= total) {
    if (n_split > 1 && split == 0 && threadIdx.x == 0) a.tc_meta[item] = make_int4(-1, 0, 0, 0);
    return;
  }
  if (before <= item && item < before + mine) {
    int64_t at = before;
    for (int b = b_first; b < b_last; ++b) {
      const int64_t n = row_tiles(load_span(a, b, false));
      if (item < at + n) {
        mi->find[0] = b;
        mi->find[1] = item - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const int seq = int(mi->find[0]);
  const SeqSpan span = load_span(a, seq, false);
  const int n_rows = span.q_len * a.group;
  const int64_t in_seq = mi->find[1], tiles = (n_rows + 255) / 256;
  const int kvh = int(in_seq % a.sh.n_kv);
  const int row0 = int(tiles - 1 - in_seq / a.sh.n_kv) * 256;  // the longest rows first
  const int rows = min(256, n_rows - row0), n_tiles_q = rows > 128 ? 2 : 1;
  if (n_split > 1 && split == 0 && threadIdx.x == 0) a.tc_meta[item] = make_int4(seq, kvh, row0, rows);
  int lo_any, hi_any, lo_all, hi_all;
  seen_range(span, row0 / a.group, a.causal, a.window, lo_any, hi_all);
  seen_range(span, (row0 + rows - 1) / a.group, a.causal, a.window, lo_all, hi_any);
  const int first = lo_any / kTile, all = max(0, (hi_any + kTile - 1) / kTile - first);
  const int j0 = first + int(int64_t(all) * split / n_split), n = first + int(int64_t(all) * (split + 1) / n_split) - j0;

  // q's rows are copied to where their operand rows will be, whole rows by
  // consecutive lanes (a thread reading its own row from global memory touches
  // 32 lines per load: 6.5 us for the operand of 256 rows, this 3).
  for (int i = threadIdx.x; i < n_tiles_q * 128 * (D / 8); i += kTcThreads) {
    const int r = i / (D / 8), piece = i % (D / 8), row = min(row0 + r, n_rows - 1), tok = row / a.group;
    cp_async16(smem_u32(sm + (r >> 7) * C::kQBytes + (piece >> 3) * kSub + sw128_off(r & 127, piece & 7)),
               a.q + int64_t(span.q0 + tok) * a.q_token + int64_t(kvh * a.group + row - tok * a.group) * a.q_head + piece * 16, 16);
  }
  cp_commit();

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[kKFull + i], 8);  // the K operand and the V exponents of the tile
      mbar_init(&bar[kKEmpty + i], n_tiles_q);
      mbar_init(&bar[kVFull + i], 4);
      mbar_init(&bar[kVEmpty + i], n_tiles_q);
      mbar_init(&bar[kAllDone + i], 1);
      mbar_init(&bar[kODone + i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar[kSFull + i], 1);
      mbar_init(&bar[kPReady + i], 4);
    }
    mbar_init(&bar[kQReady], 4 * n_tiles_q);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&mi->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  cp_wait<0>();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = mi->tmem;
  const int32_t *table = a.page_table + int64_t(seq) * a.table_stride;
  // Page-table entry and place of the 8 or 16 tokens from `tok` (page sizes are
  // multiples of 16); past the last seen token only the entry's address has to
  // be valid. The entry is looked at a tile later, so that nothing waits for it
  // here. n > 0.
  auto find_page = [&](int tok, int &entry, int &place) {
    const int p = token_page(a.sh, min(tok, hi_any - 1));
    entry = ldg_now(table + p);
    place = tok - p * a.sh.page_size;
  };

  if (warp < 8) {
    // ---- softmax: thread = row ----
    regs_up<Regs<VT>::kSoftmax>();
    const int t = warp >> 2, q4 = warp & 3, local = t * 128 + q4 * 32 + lane, row = row0 + local;
    if (t < n_tiles_q) {
      const bool live = local < rows;
      const int tok = min(row, n_rows - 1) / a.group, head = kvh * a.group + (min(row, n_rows - 1) - tok * a.group);
      int lo, hi;
      seen_range(span, tok, a.causal, a.window, lo, hi);
      float fq;  // score = fq * (kk's factor) * S
      {
        uint8_t *qs = sm + t * C::kQBytes;
        const int r = q4 * 32 + lane;
        // the row's largest magnitude, from the bits as they are
        uint32_t most = 0;
#pragma unroll
        for (int v = 0; v < D / 8; ++v) {
          const uint4 w = *reinterpret_cast<const uint4 *>(qs + (v >> 3) * kSub + sw128_off(r, v & 7));
          most = max_u16x2(max_u16x2(max_u16x2(max_u16x2(most, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu), w.z & 0x7fff7fffu), w.w & 0x7fff7fffu);
        }
        most = max(most & 0xffffu, most >> 16);
        float m = a.elem == kElemF16 ? __half2float(__ushort_as_half(uint16_t(most))) : __uint_as_float(most << 16);
        if (a.rotate) m *= 8.0f;  // H64 / 8 can make a value 8 times as large
        // 2^k brings that to [2^10, 2^11); the scale's sign goes into q
        const int k = m > 0.0f ? min(10 + 127 - int(__float_as_uint(m) >> 23), 110) : 0;
        const float up = live ? copysignf(pow2(k), a.scale_log2) : 0.0f;
        fq = fabsf(a.scale_log2) * pow2(-k);
#pragma unroll 1
        for (int h = 0; h < C::kSubs; ++h) {
          float x[64];
          load_q64(a.elem, qs + h * kSub, r, a.rotate, x);
#pragma unroll
          for (int i = 0; i < 64; ++i) x[i] = live ? x[i] * up : 0.0f;
#pragma unroll
          for (int v = 0; v < 8; ++v) {  // vector v: unit v & 3 of block v >> 2
            const int b = (v >> 2) * 32, c = v & 3;
            uint4 w;
            if constexpr (K4) {
              w.x = half2_bits(x[b + 4 * c], x[b + 4 * c + 2]);
              w.y = half2_bits(x[b + 16 + 4 * c], x[b + 16 + 4 * c + 2]);
              w.z = half2_bits(x[b + 4 * c + 1], x[b + 4 * c + 3]);
              w.w = half2_bits(x[b + 16 + 4 * c + 1], x[b + 16 + 4 * c + 3]);
            } else {
              w.x = half2_bits(x[b + 8 * c], x[b + 8 * c + 1]);
              w.y = half2_bits(x[b + 8 * c + 2], x[b + 8 * c + 3]);
              w.z = half2_bits(x[b + 8 * c + 4], x[b + 8 * c + 5]);
              w.w = half2_bits(x[b + 8 * c + 6], x[b + 8 * c + 7]);
            }
            *reinterpret_cast<uint4 *>(qs + h * kSub + sw128_off(r, v)) = w;
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kQReady]);
      }
      const uint32_t lanes = tmem + (uint32_t(q4 * 32) << 16);
      const uint32_t s_col = lanes + uint32_t(t * 128), o_col = lanes + uint32_t(256 + t * 128);
      float m = -FLT_MAX, l = 0.0f;
      int k0 = 0;
      bool ok = true;
      for (int i = 0; i < 2 * n; ++i) {  // half tiles of 64 tokens
        const int j = i >> 1, half = i & 1;
        if (!pa_wait_warp(&bar[kSFull + 2 * t + half], j & 1, spin, abort_flag, a.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t col0 = s_col + 64 * half;
        uint32_t s[2][32];
        tmem_ld32_issue(col0, s[0]);
        tmem_ld32_issue(col0 + 32, s[1]);
        // per 32 tokens: score = f S, and the V operand is in 2^-h of the first one's unit
        const volatile int *kx = mi->kx[j & 3] + 2 * half, *vx = mi->vx[j & 3] + 2 * half;
        if (i == 0) k0 = vx[0];
        const float f[2] = {fq * pow2(-kx[0]), fq * pow2(-kx[1])};
        const int h[2] = {k0 - vx[0], k0 - vx[1]};
        const int tok0 = (j0 + j) * kTile + 64 * half;
        const bool full = tok0 >= lo_all && tok0 + 64 <= hi_all;
        uint32_t p[32];
        float rm, part;
        // Weights and their sum with the maximum as it is, and the scores'
        // maximum. Straight-line code (a mask test per value would cut it into
        // dependent pieces).
        auto weigh = [&](auto masked) {
          rm = -INFINITY;
          part = 0.0f;
          tmem_ld_wait(s[0]);
          tmem_ld_wait(s[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float c0 = float(kHead + h[c]) - m;
            const uint64_t f2 = pack2(__float_as_uint(f[c]), __float_as_uint(f[c])), c2 = pack2(__float_as_uint(c0), __float_as_uint(c0));
            uint64_t sum2[2] = {0, 0};
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              uint32_t a0 = s[c][2 * k], a1 = s[c][2 * k + 1];
              if constexpr (decltype(masked)::value) {
                const int tk = tok0 + 32 * c + 2 * k;
                a0 = tk >= lo && tk < hi ? a0 : 0xff800000u;  // -infinity
                a1 = tk + 1 >= lo && tk + 1 < hi ? a1 : 0xff800000u;
              }
              m4[(2 * k) & 3] = fmaxf(m4[(2 * k) & 3], __uint_as_float(a0));
              m4[(2 * k + 1) & 3] = fmaxf(m4[(2 * k + 1) & 3], __uint_as_float(a1));
              const uint64_t x = ffma2(pack2(a0, a1), f2, c2);
              float u = __uint_as_float(uint32_t(x)), v = __uint_as_float(uint32_t(x >> 32));
              if constexpr (decltype(masked)::value) {  // where f is 0 the product of a masked score is NaN
                u = a0 == 0xff800000u ? -INFINITY : u;
                v = a1 == 0xff800000u ? -INFINITY : v;
              }
              u = ex2(u);
              v = ex2(v);
              sum2[k & 1] = fadd2(sum2[k & 1], pack2(__float_as_uint(u), __float_as_uint(v)));
              p[16 * c + k] = half2_bits(u, v);
            }
            rm = fmaxf(rm, fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), f[c], float(h[c])));
            const uint64_t both = fadd2(sum2[0], sum2[1]);
            part = fmaf(__uint_as_float(uint32_t(both)) + __uint_as_float(uint32_t(both >> 32)), pow2(-h[c]), part);
          }
        };
        for (int pass = 0; pass < 2; ++pass) {
          if (full)
            weigh(std::false_type());
          else
            weigh(std::true_type());
          const bool raise = rm > m + kRaise;
          if (!__any_sync(kFull, raise)) break;
          const float mn = raise ? rm : m, al = ex2(m - mn);
          m = mn;
          l *= al;
          if (i > 0) {
            // O is only touched once the product of the half before is done:
            // the other half's next S comes after it
            ok = pa_wait_warp(&bar[kSFull + 2 * t + (half ^ 1)], (j + half) & 1, spin, abort_flag, a.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < NB; ++c) {
              tmem_ld32(o_col + 32 * c, s[0]);
#pragma unroll
              for (int k = 0; k < 32; ++k) s[0][k] = __float_as_uint(__uint_as_float(s[0][k]) * al);
              tmem_st32(o_col + 32 * c, s[0]);
            }
          }
          tmem_ld32_issue(col0, s[0]);
          tmem_ld32_issue(col0 + 32, s[1]);
        }
        if (!ok) break;
        l += part;
        tmem_st32(col0, p);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kPReady + 2 * t + half]);
      }
      // ---- output ----
      if (ok && n > 0) ok = pa_wait_warp(&bar[kODone + t], 0, spin, abort_flag, a.err);
      if (ok) {
        tc_fence_after();
        const bool part = n_split > 1;
        const float scale = l == 0.0f ? 0.0f : part ? pow2(-k0 - kHead) : pow2(-k0) / l;
        uint8_t *out = a.o + int64_t(span.q0 + tok) * a.o_token + int64_t(head) * a.o_head;
        const int64_t pr = (item * n_split + split) * 256 + local;
#pragma unroll 1
        for (int b = 0; b < NB; ++b) {
          uint32_t v[32];
          if (n > 0) {
            tmem_ld32(o_col + 32 * b, v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0;
          }
          float y[32];  // operand row 8 i + g of the block is channel i of unit g
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < 8; ++g)
              y[V4 ? (i & 1) + 2 * g + 16 * (i >> 1) : 4 * g + i] = l == 0.0f ? 0.0f : __uint_as_float(v[8 * i + g]) * scale;
          if (live) {
            if (part) {
              float *dst = a.tc_part_o + pr * D + b * 32;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<float4 *>(dst)[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint4 w;
                if (a.elem == kElemF16) {
                  w.x = pack_pair<kElemF16>(y[8 * i], y[8 * i + 1]), w.y = pack_pair<kElemF16>(y[8 * i + 2], y[8 * i + 3]);
                  w.z = pack_pair<kElemF16>(y[8 * i + 4], y[8 * i + 5]), w.w = pack_pair<kElemF16>(y[8 * i + 6], y[8 * i + 7]);
                } else {
                  w.x = pack_pair<kElemBF16>(y[8 * i], y[8 * i + 1]), w.y = pack_pair<kElemBF16>(y[8 * i + 2], y[8 * i + 3]);
                  w.z = pack_pair<kElemBF16>(y[8 * i + 4], y[8 * i + 5]), w.w = pack_pair<kElemBF16>(y[8 * i + 6], y[8 * i + 7]);
                }
                reinterpret_cast<uint4 *>(out + b * 64)[i] = w;
              }
            }
          }
        }
        if (live) {
          if (part)
            a.tc_part_ml[pr] = make_float2(m, l * pow2(-kHead));
          else if (a.lse)
            a.lse[int64_t(span.q0 + tok) * a.n_heads + head] = l == 0.0f ? -INFINITY : (m - float(kHead) + log2f(l)) / kLog2e;
        }
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    regs_down<Regs<VT>::kOperand>();
    // ---- K operand: lane = (token of 8, unit), four groups of 8 tokens per thread ----
    const int w = warp - 8, tk = lane & 7, c = lane >> 3;
    uint32_t code[4][UK / 4], sc[4][NB / 2];
    int next[2], place[2];  // of the next tile to load (16 tokens each), asked for a tile ahead
    auto pages = [&](int j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) find_page((j0 + j) * kTile + w * 32 + 16 * h, next[h], place[h]);
    };
    // Loads have no branch around them (at its end they would be waited for):
    // where there is nothing to read, q's first bytes stand in and the scale
    // is cleared when it is used.
    uint32_t live = 0;
    auto load = [&](int j) {
      live = 0;
      bool wrong = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok0 = (j0 + j) * kTile + w * 32 + 16 * h;
        const bool want = tok0 < hi_any && tok0 + 16 > lo_any, ok = want && uint32_t(next[h]) < uint64_t(a.sh.n_pages);
        wrong = wrong || (want && !ok);
        const uint8_t *hp = a.kp.base + (int64_t(next[h]) * a.sh.n_kv + kvh) * a.kp.head_bytes;
        const uint8_t *pc = ok ? hp + ((place[h] + tk) * RBK + c * UK) : a.q;
        const uint8_t *ps = ok ? hp + a.kp.scale_off + (place[h] + tk) * (NB * 2) : a.q;
        const int code_step = ok ? 8 * RBK : 0, scale_step = ok ? 8 * NB * 2 : 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int tok = tok0 + 8 * k + tk;
          live |= uint32_t(ok && tok >= lo_any && tok < hi_any) << (2 * h + k);
          ldg_piece<UK>(pc + k * code_step, code[2 * h + k]);
          ldg_piece<NB * 2>(ps + k * scale_step, sc[2 * h + k]);
        }
      }
      if (wrong) atomicOr(a.err, kErrIndex);
      pages(j + 1);
    };
    if (n > 0) {
      pages(0);
      load(0);
    }
    for (int j = 0; j < n; ++j) {
      uint32_t e = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < NB / 2; ++k) {
          sc[i][k] = live >> i & 1 ? sc[i][k] : 0;
          e = max_u16x2(e, sc[i][k]);
        }
      const int kk = scale_up(e);
      if (!pa_wait_warp(&bar[kKEmpty + (j & 1)], ((j >> 1) & 1) ^ 1, spin, abort_flag, a.err)) break;
      if (lane == 0) mi->kx[j & 3][w] = kk;
      const uint32_t up = half2_pow2(kk);
      uint8_t *ks = sm + C::kOffK + (j & 1) * C::kKBytes;
      // Two groups of tokens per turn: unrolled over all four, the roles' loops
      // no longer fit the instruction cache together (8-bit K: 309 -> 277 us
      // per prompt chunk of 2048 tokens at 8192).
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = w * 32 + turn * 16 + i * 8 + tk;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t d = hmul2(sc[i][b / 2], up), d2 = __byte_perm(d, d, (b & 1) ? 0x3232 : 0x1010);
            uint4 v;
            if constexpr (K4) {
              const uint32_t x = code[i][b], y = x >> 8;
              v = make_uint4(hmul2(codes4_lo(x), d2), hmul2(codes4_hi(x), d2), hmul2(codes4_lo(y), d2), hmul2(codes4_hi(y), d2));
            } else {
              const uint2 x = codes_to_f16x2(code[i][2 * b]), y = codes_to_f16x2(code[i][2 * b + 1]);
              v = make_uint4(hmul2(x.x, d2), hmul2(x.y, d2), hmul2(y.x, d2), hmul2(y.y, d2));
            }
            *reinterpret_cast<uint4 *>(ks + (b >> 1) * kSub + sw128_off(r, (b & 1) * 4 + c)) = v;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int k = 0; k < UK / 4; ++k) code[i][k] = code[i + 2][k];
#pragma unroll
          for (int k = 0; k < NB / 2; ++k) sc[i][k] = sc[i + 2][k];
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[kKFull + (j & 1)]);
      if (j + 1 < n) load(j + 1);
    }
  } else if (warp < 16) {
    regs_down<Regs<VT>::kOperand>();
    // ---- V operand, transposed: thread = (8 tokens, unit g): 8 tokens of 4 channels per block ----
    const int w = warp - 12, g = lane & 7, grp = w * 4 + (lane >> 3);
    uint32_t code[8][(UV + 3) / 4], sc[8][NB / 2];
    int next = 0, place = 0;  // of the next tile to load
    auto pages = [&](int j) { find_page((j0 + j) * kTile + grp * 8, next, place); };
    uint32_t live = 0;
    auto load = [&](int j) {  // no branch around the loads, as for K
      const int tok0 = (j0 + j) * kTile + grp * 8;
      const bool want = tok0 < hi_any && tok0 + 8 > lo_any, ok = want && uint32_t(next) < uint64_t(a.sh.n_pages);
      if (want && !ok) atomicOr(a.err, kErrIndex);
      const uint8_t *hp = a.vp.base + (int64_t(next) * a.sh.n_kv + kvh) * a.vp.head_bytes;
      const uint8_t *pc = ok ? hp + place * RBV + g * UV : a.q, *ps = ok ? hp + a.vp.scale_off + place * NB * 2 : a.q;
      const int sc_step = ok ? NB * 2 : 0, code_step = ok ? RBV : 0;
      live = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        live |= uint32_t(ok && tok0 + i >= lo_any && tok0 + i < hi_any) << i;
        ldg_piece<UV>(pc + i * code_step, code[i]);
        ldg_piece<NB * 2>(ps + i * sc_step, sc[i]);
      }
      pages(j + 1);
    };
    if (n > 0) {
      pages(0);
      load(0);
    }
    for (int j = 0; j < n; ++j) {
      uint32_t e = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < NB / 2; ++k) {
          sc[i][k] = live >> i & 1 ? sc[i][k] : 0;
          e = max_u16x2(e, sc[i][k]);
        }
      const int ve = scale_up(e);
      // kVEmpty of the first two tiles lets this warp get to tile 2 before a K
      // warp has arrived for tile 0: without the wait it would count in its
      // place, and S of tile 0 be taken from rows not written yet. Nearly
      // always complete.
      if (!pa_wait_warp(&bar[kKFull + (j & 1)], ((j >> 1) & 1) ^ 1, spin, abort_flag, a.err)) break;
      if (lane == 0) {
        mi->vx[j & 3][w] = ve;
        mbar_arrive(&bar[kKFull + (j & 1)]);
      }
      if (!pa_wait_warp(&bar[kVEmpty + (j & 1)], ((j >> 1) & 1) ^ 1, spin, abort_flag, a.err)) break;
      const uint32_t up = half2_pow2(ve);
      uint8_t *vs = sm + C::kOffV + (j & 1) * C::kVBytes + (grp >> 3) * C::kVSub;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t o[4][4];  // [channel of the unit][token pair]
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t d2 = hmul2(__byte_perm(sc[2 * k][b / 2], sc[2 * k + 1][b / 2], (b & 1) ? 0x7632 : 0x5410), up);
          if constexpr (V4) {
            const uint32_t x = __byte_perm(code[2 * k][b / 2], code[2 * k + 1][b / 2], (b & 1) ? 0x7632 : 0x5410), y = x >> 8;
            o[0][k] = hmul2(codes4_lo(x), d2);  // channel 2g
            o[1][k] = hmul2(codes4_lo(y), d2);  // 2g + 1
            o[2][k] = hmul2(codes4_hi(x), d2);  // 16 + 2g
            o[3][k] = hmul2(codes4_hi(y), d2);
          } else {
            const uint32_t w0 = code[2 * k][b], w1 = code[2 * k + 1][b];
            const uint2 x = codes_to_f16x2(__byte_perm(w0, w1, 0x5140)), y = codes_to_f16x2(__byte_perm(w0, w1, 0x7362));
            o[0][k] = hmul2(x.x, d2), o[1][k] = hmul2(x.y, d2), o[2][k] = hmul2(y.x, d2), o[3][k] = hmul2(y.y, d2);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4 *>(vs + sw128_off(b * 32 + 8 * i + g, grp & 7)) = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[kVFull + (j & 1)]);
      if (j + 1 < n) load(j + 1);
    }
  } else {
    regs_down<Regs<VT>::kIssue>();
    const int t = warp - 16;
    if (t < n_tiles_q && lane == 0) {
      // ---- MMA issue, a warp per row tile ----
      // Operand descriptors differ in their low words' address field only (in
      // 16 bytes, below 2^14): one 32-bit addition per product.
      const uint64_t d0 = sw128_desc(smem_u32(sm));
      const uint32_t lo0 = uint32_t(d0), hi0 = uint32_t(d0 >> 32);
      auto desc = [&](uint32_t offset) { return pack2(lo0 + (offset >> 4), hi0); };
      // S of half h of tile j
      auto issue_s = [&](int h, int j) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = (k >> 2) * kSub + (k & 3) * 32;
          tc_mma(tmem + uint32_t(t * 128 + h * 64), desc(t * C::kQBytes + at),
                 desc(C::kOffK + (j & 1) * C::kKBytes + h * (kSub / 2) + at), kIdescS, k > 0);
        }
        tc_commit(&bar[kSFull + 2 * t + h]);
      };
      bool ok = n > 0 && pa_wait(&bar[kQReady], 0, spin, abort_flag, a.err) && pa_wait(&bar[kKFull], 0, spin, abort_flag, a.err);
      if (ok) {
        tc_fence_after();
        issue_s(0, 0);
        issue_s(1, 0);
        tc_commit(&bar[kKEmpty]);
      }
      // A wait holds up the products behind it even where its phase is long
      // complete, so a step's operands are tested for while the products of
      // the step before are queued.
      auto operands = [&](auto look, int j) {
        return look(&bar[kVFull + (j & 1)], (j >> 1) & 1) && (j + 1 >= n || look(&bar[kKFull + ((j + 1) & 1)], ((j + 1) >> 1) & 1));
      };
      bool seen = false;
      for (int j = 0; j < n && ok; ++j) {
        const bool more = j + 1 < n;
        if (!seen)
          ok = operands([&](uint64_t *b, uint32_t parity) { return pa_wait(b, parity, spin, abort_flag, a.err); }, j);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || !(ok = pa_wait(&bar[kPReady + 2 * t + h], j & 1, spin, abort_flag, a.err))) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_ts(tmem + uint32_t(256 + t * 128), tmem + uint32_t(t * 128 + h * 64 + k * 8),
                      desc(C::kOffV + (j & 1) * C::kVBytes + h * C::kVSub + k * 32), kIdescO, j > 0 || h > 0 || k > 0);
          if (h == 1) tc_commit(&bar[kVEmpty + (j & 1)]);
          if (h == 1 && more) seen = operands([](uint64_t *b, uint32_t parity) { return mbar_test_wait(b, parity); }, j + 1);
          if (more) {
            issue_s(h, j + 1);
            if (h == 1) tc_commit(&bar[kKEmpty + ((j + 1) & 1)]);
          } else if (h == 0) {
            tc_commit(&bar[kSFull + 2 * t]);  // no S: the product is done
          } else {
            tc_commit(&bar[kODone + t]);
          }
        }
      }
      tc_commit(&bar[kAllDone + t]);
      tc_drain(&bar[kAllDone + t], 0);
    }
  }
  __syncthreads();
  if (warp == 16) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int NB, int KT, int VT>
cudaError_t launch_one(const PagedAttnArgs &a, int64_t items, int n_split, cudaStream_t stream) {
  cudaError_t e = ensure_smem(reinterpret_cast<const void *>(k_paged_tc<NB, KT, VT>), TcCfg<NB>::kSmem);
  if (e != cudaSuccess) return e;
  k_paged_tc<NB, KT, VT><<<unsigned(items * n_split), kTcThreads, TcCfg<NB>::kSmem, stream>>>(a, n_split, spin_limit());
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tc(const PagedAttnArgs &a, int64_t items, int n_split, cudaStream_t stream) {
  return by_cache_types(a.kt, a.vt, [&](auto k, auto v) {
    return a.sh.nb == 4 ? launch_one<4, k.value, v.value>(a, items, n_split, stream)
                        : launch_one<2, k.value, v.value>(a, items, n_split, stream);
  });
}

}  // namespace paged
}  // namespace bq

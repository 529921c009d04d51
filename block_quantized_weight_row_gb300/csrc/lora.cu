// lora.cu — low-rank adapters of many requests beside a shared projection
// (include/bq.h: bq_lora):  out_t = y_t + s_a B_a (A_a x_t),  a = adapter[t].
//
// Bound by memory: 2 r (K + M) products per token against a row of x, y and out
// each (r is 8 to 128), and in a decode step the adapters' own 2 r (K + M) bytes.
// Tokens of one adapter are brought together in tiles of 16 or 64 tokens, so that
// an adapter is read once per tile and the products run on tensor instructions:
//   1. k_lora_group (from kLeaders tokens on): tokens sorted by adapter, and the
//      list of tiles. Below that every CTA finds its tile itself: the tokens of
//      the adapter of token j, if j is the first of sixteen of them.
//   2. H[t] = s_a A_a x_t, K cut over the warps and the CTAs of a cluster, whose
//      sums meet in shared memory in a fixed order: k_lora_shrink16 and 64 on
//      warp-level instructions, k_lora_shrink_tc on tcgen05 (lora_tc.cu).
//   3. out_t = y_t + B_a H[t]: k_lora_expand for tiles of 16, k_lora_expand_tc on
//      tcgen05 for tiles of 64.
// Measured (GPU alone): 48 fp32 tokens of 16 adapters, 4096 to 4096 at rank 16, 10.2
// to 10.6 us; 8192 bf16 tokens, 4096 to 11008 fp32 columns at rank 64, 163.5 us (8 for step
// 1, 29, and 128 for 720 MB of y and out: 5.6 TB/s).
// A tile's rows do not depend on one another, so neither the order inside an
// adapter nor the other tokens change a result.
//
// Fragments come straight from global memory, 16 bytes per lane: a product's sum
// over k may be taken in any order, so lane t of a quad gives its instruction the
// 8 consecutive k 8t .. 8t + 7 of 32 in place of the pairs of its layout, of both
// operands alike. For the second product the columns are permuted too, so that a
// lane's results over four n-tiles are whole 16-byte pieces of out.
//
// Terms. A 16-bit row meets adapters of its own type: products are exact. An fp32
// row beside bf16 adapters is cut into three bf16 terms (its 24 bits, exact),
// beside fp16 ones into two tf32 terms (22 bits; fp16 is exact in tf32). H is kept
// in fp32 and enters the second product in bf16 terms, three for fp32 rows of out
// and two (16 bits) for bf16 ones, or in two fp16 terms (22 bits) after scaling
// each row by a power of two to at most 2^15.
#include <algorithm>

#include "lora.cuh"

namespace bq {
namespace {

constexpr int kGroupThreads = 1024, kShrinkThreads = 128, kExpandThreads = 256;

// ----------------------------------------------------------------- group --

template <int TM>
__global__ void __launch_bounds__(kGroupThreads) k_lora_group(const LoraArgs a, const LoraWork w) {
  __shared__ int count[kMaxBins], tile0[kMaxBins + 1];
  __shared__ int sums[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bins = a.n_adapters + 1;
  pdl_launch_dependents();
  for (int b = tid; b < bins; b += kGroupThreads) count[b] = 0;
  __syncthreads();
  // the loads of kIds rounds are in flight together; whole warps, as the votes need them
  constexpr int kIds = 4;
  auto each = [&](auto f) {
#pragma unroll 1
    for (int t0 = tid; t0 - tid < a.n_tokens; t0 += kIds * kGroupThreads) {
      int id[kIds];
#pragma unroll
      for (int i = 0; i < kIds; ++i) id[i] = t0 + i * kGroupThreads < a.n_tokens ? __ldg(a.adapter + t0 + i * kGroupThreads) : -1;
#pragma unroll
      for (int i = 0; i < kIds; ++i) {
        const int t = t0 + i * kGroupThreads;
        const int bin = t >= a.n_tokens ? -1 : uint32_t(id[i]) < uint32_t(a.n_adapters) ? id[i] + 1 : 0;
        // tokens in runs: one atomic for a warp; else one per token, whose collisions are few
        f(t, id[i], bin, __all_sync(kFull, bin == __shfl_sync(kFull, bin, 0)));
      }
    }
  };
  bool bad = false;
  each([&](int, int id, int bin, bool all) {
    bad |= bin == 0 && id != -1;
    if (bin >= 0 && (lane == 0 || !all)) atomicAdd(&count[bin], all ? 32 : 1);
  });
  if (bad) atomicOr(a.err, kErrIndex);
  __syncthreads();
  // exclusive sums over the bins of tokens and of tiles, a run of bins per thread
  const int run = (bins + kGroupThreads - 1) / kGroupThreads, b0 = min(tid * run, bins), b1 = min(b0 + run, bins);
  int n = 0, m = 0;
  for (int b = b0; b < b1; ++b) n += count[b], m += (count[b] + TM - 1) / TM;
  int ni = n, mi = m;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(kFull, ni, d), y = __shfl_up_sync(kFull, mi, d);
    if (lane >= d) ni += x, mi += y;
  }
  if (lane == 31) sums[0][warp] = ni, sums[1][warp] = mi;
  __syncthreads();
  ni -= n, mi -= m;
  // the warps before this one: their sums by a reduction over the lanes, 32 as the warps are (777 tokens: 17.2 -> 16.6 us for the call)
  ni += __reduce_add_sync(kFull, lane < warp ? sums[0][lane] : 0);
  mi += __reduce_add_sync(kFull, lane < warp ? sums[1][lane] : 0);
  for (int b = b0; b < b1; ++b) {
    const int c = count[b];
    tile0[b] = mi;
    count[b] = ni;  // from here on: where the bin's next token goes
    ni += c, mi += (c + TM - 1) / TM;
  }
  if (tid == kGroupThreads - 1) tile0[bins] = mi;  // the last thread's sums end with all
  __syncthreads();
  const int tiles = tile0[bins];
  if (tid == 0) *w.n_tiles = tiles;
  for (int i = tid; i < tiles; i += kGroupThreads) {
    int lo = 0, hi = bins;  // the last bin with tile0 <= i that has tiles
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      (tile0[mid] <= i ? lo : hi) = mid;
    }
    const int first = count[lo] + (i - tile0[lo]) * TM, end = lo + 1 < bins ? count[lo + 1] : a.n_tokens;
    w.tiles[i] = LoraTile{lo - 1, first, min(TM, end - first), 0};
  }
  __syncthreads();
  each([&](int t, int, int bin, bool all) {
    int at = 0;
    if (bin >= 0 && (lane == 0 || !all)) at = atomicAdd(&count[bin], all ? 32 : 1);
    if (all) at = __shfl_sync(kFull, at, 0) + lane;
    if (bin >= 0) w.sorted[at] = t;
  });
}

// -------------------------------------------------------------- products --

template <int WE>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (WE == kElemBF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// fp32 bits rounded to tf32 (11 significant bits)
__device__ __forceinline__ uint32_t to_tf32(uint32_t x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(__uint_as_float(x)));
  return r;
}

// 32 k of a row: a lane's 8 of them
template <int XE>
struct RowWords {
  uint4 v[XE == kElemF32 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t *p) {
    v[0] = __ldg(reinterpret_cast<const uint4 *>(p));
    if constexpr (XE == kElemF32) v[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
  }
};

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// acc[nt] += x (rows g, g + 8; 32 k) times A (n-tile nt; 32 k)
template <int XE, int WE, int NT>
__device__ __forceinline__ void shrink_step(float (&acc)[NT][4], const RowWords<XE> &lo, const RowWords<XE> &hi, const uint4 (&bw)[NT]) {
  if constexpr (XE != kElemF32) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma16<WE>(acc[nt], lo.v[0].x, hi.v[0].x, lo.v[0].y, hi.v[0].y, bw[nt].x, bw[nt].y);
      mma16<WE>(acc[nt], lo.v[0].z, hi.v[0].z, lo.v[0].w, hi.v[0].w, bw[nt].z, bw[nt].w);
    }
  } else if constexpr (WE == kElemBF16) {
    float l[8], h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = __uint_as_float(word(lo.v[i >> 2], i & 3)), h[i] = __uint_as_float(word(hi.v[i >> 2], i & 3));
    uint32_t lw[3][4], hw[3][4];
#pragma unroll
    for (int term = 0; term < 3; ++term)
#pragma unroll
      for (int i = 0; i < 4; ++i) lw[term][i] = cut_pair(l[2 * i], l[2 * i + 1]), hw[term][i] = cut_pair(h[2 * i], h[2 * i + 1]);
#pragma unroll
    for (int term = 2; term >= 0; --term)  // the smallest first: nothing large is there yet for the adder to align them to
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma16<WE>(acc[nt], lw[term][0], hw[term][0], lw[term][1], hw[term][1], bw[nt].x, bw[nt].y);
        mma16<WE>(acc[nt], lw[term][2], hw[term][2], lw[term][3], hw[term][3], bw[nt].z, bw[nt].w);
      }
  } else {
    uint32_t l[2][8], h[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = word(lo.v[i >> 2], i & 3), y = word(hi.v[i >> 2], i & 3);
      l[0][i] = to_tf32(x), h[0][i] = to_tf32(y);
      l[1][i] = to_tf32(__float_as_uint(__fsub_rn(__uint_as_float(x), __uint_as_float(l[0][i]))));
      h[1][i] = to_tf32(__float_as_uint(__fsub_rn(__uint_as_float(y), __uint_as_float(h[0][i]))));
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 b = unpack_pair<kElemF16>(word(bw[nt], i));
#pragma unroll
        for (int term = 1; term >= 0; --term)
          mma_tf32(acc[nt], l[term][2 * i], h[term][2 * i], l[term][2 * i + 1], h[term][2 * i + 1], __float_as_uint(b.x), __float_as_uint(b.y));
      }
  }
}

// total += acc, acc = 0: the tensor instructions' adder truncates, so chains are kept short (in
// k_lora_shrink16 a block of 32 k: 48 fp32 tokens at K = 4096 and rank 16 are off by 1e-7 of the output's
// norm, by 4.2e-7 with four blocks and the terms in the order of their cutting; 2.7e-7 in fp32 sums; 10.3 us for 10.2)
template <int NT>
__device__ __forceinline__ void take(float (&total)[NT][4], float (&acc)[NT][4]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) total[nt][i] += acc[nt][i], acc[nt][i] = 0.0f;
}
template <int NT>
__device__ __forceinline__ void put(float *part, const float (&v)[NT][4], int g, int t) {  // a warp's 16 rows, in pairs
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    *reinterpret_cast<float2 *>(part + g * (8 * NT) + nt * 8 + 2 * t) = make_float2(v[nt][0], v[nt][1]);
    *reinterpret_cast<float2 *>(part + (g + 8) * (8 * NT) + nt * 8 + 2 * t) = make_float2(v[nt][2], v[nt][3]);
  }
}

// Tiles of 16 tokens, up to 32 ranks of the adapter (NT n-tiles of 8; other
// clusters have its others, so that ranks, too, are spread over the SMs). Each warp
// has all of the tile's tokens and a quarter of the CTA's k, and loads its operands
// itself: in a decode step a warp has up to four blocks of 32 k, all in flight at once.
template <int XE, int WE, int NT>
__global__ void __launch_bounds__(kShrinkThreads) k_lora_shrink16(const LoraArgs a, const LoraWork w, const int splits) {
  __shared__ __align__(16) float part[4][16][8 * NT];
  __shared__ int rows[16];
  constexpr int XS = Elem<XE>::kBytes;
  constexpr int kAhead = 4;  // blocks in flight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  if (w.sorted) {
    pdl_wait();
  } else if (threadIdx.x == 0 && blockIdx.x == 0) {
    const int id = __ldg(a.adapter + blockIdx.y);
    if (id < -1 || id >= a.n_adapters) atomicOr(a.err, kErrIndex);
  }
  int ad, count;
  if (!find_tile<16>(a, w, blockIdx.y, rows, ad, count) || ad < 0) return;  // all CTAs of the cluster alike
  const int nb = a.K / 32, split = blockIdx.x % splits, first = int(blockIdx.x) / splits * 8 * NT, pieces = splits * 4, piece = split * 4 + warp;
  const int k0 = int(int64_t(nb) * piece / pieces), k1 = int(int64_t(nb) * (piece + 1) / pieces);
  const uint8_t *lo = a.x + rows[g] * a.x_row + t * 8 * XS, *hi = a.x + rows[g + 8] * a.x_row + t * 8 * XS;
  const uint8_t *ap = a.A + (int64_t(ad) * a.rank + first + g) * a.K * 2 + t * 16;
  const bool high = count > 8;
  float acc[NT][4] = {}, total[NT][4] = {};
  for (int k = k0; k < k1; k += kAhead) {
    RowWords<XE> xl[kAhead], xh[kAhead];
    uint4 bw[kAhead][NT];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (k + u < k1) {
        xl[u].load(lo + int64_t(k + u) * 32 * XS);
        xh[u] = xl[u];
        if (high) xh[u].load(hi + int64_t(k + u) * 32 * XS);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          bw[u][nt] = make_uint4(0, 0, 0, 0);
          if (first + nt * 8 < a.rank) bw[u][nt] = __ldg(reinterpret_cast<const uint4 *>(ap + (int64_t(nt) * 8 * a.K + (k + u) * 32) * 2));
        }
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (k + u < k1) {
        shrink_step<XE, WE, NT>(acc, xl[u], xh[u], bw[u]);
        take(total, acc);
      }
  }
  put<NT>(&part[warp][0][0], total, g, t);
  sum_tile<4>(a, w, &part[0][0][0], 8 * NT, 16 * 8 * NT, rows, ad, count, first, min(8 * NT, a.rank - first), split, splits);
}

// Tiles of 64 tokens on warp-level instructions, up to 64 ranks: 16-bit rows of up
// to 64 ranks (28 to 31 us for 8192 bf16 tokens of 4096 at rank 64, where the kernel of
// lora_tc.cu takes 32 to 35; at rank 16 21) and fp32 rows beside fp16 adapters (which that
// kernel cannot take: terms of fp16 would need each row's range first). Each of the
// four warps has 16 of the tokens and all of the CTA's k. Rows of x and of the
// adapter come through a ring of stages of 64 k by asynchronous copies (straight
// loads left a warp waiting for memory in every block of 32 k: 60 us for 2048 tokens).
// A stage: two blocks of 32 k, each a row of 64 bytes per token and rank (fp32
// rows: 128 bytes, the even 16-byte pieces in one half, which half alternates
// from row to row), so that a quarter-warp's reads of two rows meet no bank twice.
template <int XE, int NT>
struct Ring {
  static constexpr int kStages = 3;
  static constexpr int kXRow = 32 * Elem<XE>::kBytes, kXBlock = 64 * kXRow, kABlock = 8 * NT * 64;
  static constexpr int kStage = 2 * (kXBlock + kABlock);
  static constexpr int kBytes = kStages * kStage > 64 * 8 * NT * 4 ? kStages * kStage : 64 * 8 * NT * 4;  // or the sums, afterwards
};

template <int XE, int WE, int NT>
__global__ void __launch_bounds__(kShrinkThreads) k_lora_shrink64(const LoraArgs a, const LoraWork w, const int splits) {
  using R = Ring<XE, NT>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int rows[64];
  constexpr int XS = Elem<XE>::kBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  pdl_wait();
  int ad, count;
  if (!find_tile<64>(a, w, blockIdx.y, rows, ad, count) || ad < 0) return;  // all CTAs of the cluster alike
  const int nb = a.K / 32, split = blockIdx.x % splits, first = int(blockIdx.x) / splits * 8 * NT;
  const int k0 = int(int64_t(nb) * split / splits), k1 = int(int64_t(nb) * (split + 1) / splits);
  const int stages = (k1 - k0 + 1) / 2;
  // a thread copies one 16-byte piece of every kStep-th row; rows without a
  // token (or a rank) are left out: what they hold reaches only their own sums
  constexpr int kPieces = 2 * R::kXRow / 16, kStep = kShrinkThreads / kPieces, kRows = 64 / kStep;
  const int xp = tid % kPieces, xr = tid / kPieces, xb = xp / (kPieces / 2), xc = xp % (kPieces / 2);
  const uint8_t *src[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) src[i] = a.x + rows[xr + i * kStep] * a.x_row + (int64_t(k0) * 32) * XS + xp * 16;
  const int ap = tid % 8, ar = tid / 8;  // 8 pieces of 64 k, 16 ranks at a time
  const uint8_t *asrc = a.A + (int64_t(ad) * a.rank + first + ar) * a.K * 2 + int64_t(k0) * 64 + ap * 16;
  auto fill = [&](int s) {
    uint8_t *x = ring + (s % R::kStages) * R::kStage, *ad_rows = x + 2 * R::kXBlock;
    if (k0 + 2 * s + xb < k1) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = xr + i * kStep;
        const int at = XE == kElemF32 ? (xc >> 1) + 4 * ((xc & 1) ^ (r & 1)) : xc;
        if (r < count) copy16(x + xb * R::kXBlock + r * R::kXRow + at * 16, src[i] + int64_t(s) * 64 * XS);
      }
    }
    if (k0 + 2 * s + ap / 4 < k1) {
#pragma unroll
      for (int i = 0; i < (NT + 1) / 2; ++i) {
        const int r = ar + 16 * i;
        if (r < 8 * NT && first + r < a.rank) copy16(ad_rows + (ap / 4) * R::kABlock + r * 64 + (ap % 4) * 16, asrc + (int64_t(i) * 16 * a.K + s * 64) * 2);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < R::kStages - 1; ++s) {
    if (s < stages)
      fill(s);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const int r0 = warp * 16;
  const bool idle = r0 >= count;  // no token in this warp's rows
  float acc[NT][4] = {}, total[NT][4] = {};
  for (int s = 0; s < stages; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(R::kStages - 2) : "memory");
    __syncthreads();  // the stage is there, and the one before it is used up
    if (s + R::kStages - 1 < stages)
      fill(s + R::kStages - 1);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
    if (!idle) {
      const uint8_t *x = ring + (s % R::kStages) * R::kStage, *ad_rows = x + 2 * R::kXBlock;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (k0 + 2 * s + b >= k1) break;
        RowWords<XE> xl, xh;
        uint4 bw[NT];
        const uint8_t *pl = x + b * R::kXBlock + (r0 + g) * R::kXRow, *ph = pl + 8 * R::kXRow;
        if constexpr (XE == kElemF32) {
          const int half = (g & 1) * 64 + t * 16;  // rows g and g + 8 are both even or both odd
          xl.v[0] = *reinterpret_cast<const uint4 *>(pl + half);
          xl.v[1] = *reinterpret_cast<const uint4 *>(pl + (half ^ 64));
          xh.v[0] = *reinterpret_cast<const uint4 *>(ph + half);
          xh.v[1] = *reinterpret_cast<const uint4 *>(ph + (half ^ 64));
        } else {
          xl.v[0] = *reinterpret_cast<const uint4 *>(pl + t * 16);
          xh.v[0] = *reinterpret_cast<const uint4 *>(ph + t * 16);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) bw[nt] = *reinterpret_cast<const uint4 *>(ad_rows + b * R::kABlock + (nt * 8 + g) * 64 + t * 16);
        shrink_step<XE, WE, NT>(acc, xl, xh, bw);
      }
      // after 16 instructions of fp32 rows (32: 600 of 4096 at rank 64 off by 4.7e-7 of the output's norm for 2.8e-7), 8 in 16 bits
      if (XE == kElemF32 || (s & 1)) take(total, acc);
    }
  }
  take(total, acc);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // the ring becomes the sums' place
  float *part = reinterpret_cast<float *>(ring);
  put<NT>(part + r0 * (8 * NT), total, g, t);
  sum_tile<1>(a, w, part, 8 * NT, 0, rows, ad, count, first, min(8 * NT, a.rank - first), split, splits);
}

// ---------------------------------------------------------------- expand --

// A lane's 8 columns of a turn's 32 are pieces of 16 bytes, a row's four lanes
// side by side in one access, so that it covers whole sectors: 8 columns from 8 t
// (16-bit rows), or 4 from 4 t and 4 from 16 + 4 t (fp32).
template <int YE>
struct Piece {
  static constexpr int kCount = Elem<YE>::kBytes / 2, kCols = 8 / kCount;
  static __device__ __forceinline__ int column(int k, int t) { return 16 * k + kCols * t; }
  // column c of n-tile j (a lane has 2 t and 2 t + 1 of each): the lane's column 2 j + c % 2
  static __device__ __forceinline__ int tile_column(int j, int c) {
    const int i = 2 * j + (c & 1);
    return column(i / kCols, c >> 1) + i % kCols;
  }
};

// one piece: from 16 bytes, or its first n columns one by one
template <int YE>
__device__ __forceinline__ void read_y(const uint8_t *p, float *v) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (YE == kElemF32) {
      v[i] = __uint_as_float(word(a, i));
    } else {
      const float2 f = unpack_pair<YE>(word(a, i));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
template <int YE>
__device__ __forceinline__ void load_y(const uint8_t *p, int n, float *v) {
#pragma unroll
  for (int i = 0; i < Piece<YE>::kCols; ++i)
    if (i < n) {
      if constexpr (YE == kElemF32) v[i] = reinterpret_cast<const float *>(p)[i];
      if constexpr (YE == kElemF16) v[i] = __half2float(reinterpret_cast<const __half *>(p)[i]);
      if constexpr (YE == kElemBF16) v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
    }
}
template <int YE>
__device__ __forceinline__ void store_y(uint8_t *p, int n, bool vec, const float *v) {
  if (vec && n >= Piece<YE>::kCols) {
    if constexpr (YE == kElemF32)
      __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    else
      __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_pair<YE>(v[0], v[1]), pack_pair<YE>(v[2], v[3]), pack_pair<YE>(v[4], v[5]), pack_pair<YE>(v[6], v[7])));
  } else {
#pragma unroll
    for (int i = 0; i < Piece<YE>::kCols; ++i)
      if (i < n) {
        if constexpr (YE == kElemF32) reinterpret_cast<float *>(p)[i] = v[i];
        if constexpr (YE == kElemF16) reinterpret_cast<__half *>(p)[i] = __float2half_rn(v[i]);
        if constexpr (YE == kElemBF16) reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v[i]);
      }
  }
}

template <int WE, int YE, int KB>
struct Expand {
  static constexpr int kTerms = WE == kElemF16 ? 2 : YE == kElemF32 ? 3 : 2;
  static constexpr int kPitch = KB == 1 ? 64 : KB * 64 + 64;  // 64 modulo 128: a quarter-warp's 16-byte reads of two rows meet no bank twice
  static constexpr int kPieces = 2 * Elem<YE>::kBytes / 2;  // 16-byte pieces of y per lane and turn
  static constexpr int kTermBytes = kTerms * 16 * kPitch, kYBytes = kPieces * 512;
  static constexpr int kBytes = kTermBytes + (kExpandThreads / 32) * 2 * kYBytes;
  static_assert(KB == 1 || KB % 2 == 0, "pitch");
};

// Tiles of 16 tokens; KB: blocks of 32 ranks. A warp has the tile's tokens and 32
// columns a turn, the CTA's 8 warps 256. A lane's pieces of y come a turn ahead,
// by asynchronous copies into places of its own (nobody else waits for them); the
// first turn's, and its part of B, are asked for before the launch before this one
// has ended.
template <int WE, int YE, int KB>
__global__ void __launch_bounds__(kExpandThreads, 2) k_lora_expand(const LoraArgs a, const LoraWork w, const int turns) {
  using E = Expand<WE, YE, KB>;
  constexpr int TM = 16, kStep = 256, kTerms = E::kTerms, kPitch = E::kPitch;
  using Pc = Piece<YE>;
  constexpr int YS = Elem<YE>::kBytes, kPer = Pc::kCount;
  constexpr int kAhead = KB < 2 ? KB : 2;              // blocks of B in flight
  extern __shared__ __align__(16) uint8_t terms[];     // [term][row], rows of kPitch bytes; then y
  __shared__ float unscale[TM];
  __shared__ int rows[TM];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  if (w.sorted) pdl_wait();
  int ad, count;
  if (!find_tile<TM>(a, w, blockIdx.y, rows, ad, count)) return;
  if (ad < 0 && a.y == a.out) {
    // every launch has a tile that waits for the one before it, so that it never ends before that one
    if (!w.sorted) pdl_wait();
    return;
  }
  uint8_t *const mine = terms + E::kTermBytes + warp * 2 * E::kYBytes + lane * 16;
  const int first = int(blockIdx.x) * turns * kStep + warp * 32;  // column of the first turn
  // y's pieces of a turn; rows of another alignment and the last columns are loaded when they are needed
  auto ask = [&](int turn) {
    const int m0 = first + turn * kStep;
    if (a.y && a.y_vec && turn < turns) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (8 * h + g < count) {
          const uint8_t *p = a.y + rows[8 * h + g] * a.y_row;
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int c = m0 + Pc::column(k, t);
            if (c + Pc::kCols <= a.M) copy16(mine + (turn & 1) * E::kYBytes + (h * kPer + k) * 512, p + int64_t(c) * YS);
          }
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto load_b = [&](uint4 (&bw)[4], int m0, int kb) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // column g of n-tile j
      const int m = m0 + Pc::tile_column(j, g);
      bw[j] = make_uint4(0, 0, 0, 0);
      if (ad >= 0 && m < a.M && kb * 32 + 8 * t < a.rank)
        bw[j] = __ldg(reinterpret_cast<const uint4 *>(a.B + ((int64_t(ad) * a.M + m) * a.rank + kb * 32 + 8 * t) * 2));
    }
  };
  ask(0);
  uint4 bw[kAhead][4];
#pragma unroll
  for (int kb = 0; kb < kAhead; ++kb) load_b(bw[kb], first, kb);
  if (!w.sorted) pdl_wait();
  if (ad >= 0) {
    for (int r = warp; r < TM; r += kExpandThreads / 32) {
      float h[KB], m = 0.0f;
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        const int c = lane + 32 * i;
        h[i] = r < count && c < a.rank ? __ldcg(w.H + int64_t(rows[r]) * a.rank + c) : 0.0f;
        m = fmaxf(m, fabsf(h[i]));
      }
      float up = 1.0f;
      if constexpr (WE == kElemF16) up = scale_row(m, unscale, r, lane);
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        float x = h[i] * up;
#pragma unroll
        for (int k = 0; k < kTerms; ++k) {
          uint16_t *to = reinterpret_cast<uint16_t *>(terms + (k * TM + r) * kPitch + (lane + 32 * i) * 2);
          if constexpr (WE == kElemF16) {
            const __half f = __float2half_rn(x);
            *to = __half_as_ushort(f);
            x -= __half2float(f);
          } else {
            const __nv_bfloat16 f = __float2bfloat16_rn(x);
            *to = __bfloat16_as_ushort(f);
            x -= __bfloat162float(f);
          }
        }
      }
    }
    __syncthreads();
  }
  for (int turn = 0; turn < turns; ++turn) {
    const int m0 = first + turn * kStep;
    if (m0 >= a.M) break;
    ask(turn + 1);
    float acc[4][4] = {};
    if (ad >= 0) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        uint4(&b)[4] = bw[kb % kAhead];
#pragma unroll
        for (int k = kTerms - 1; k >= 0; --k) {
          const uint4 lo = *reinterpret_cast<const uint4 *>(terms + (k * TM + g) * kPitch + kb * 64 + 16 * t);
          const uint4 hi = *reinterpret_cast<const uint4 *>(terms + (k * TM + g + 8) * kPitch + kb * 64 + 16 * t);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma16<WE>(acc[j], lo.x, hi.x, lo.y, hi.y, b[j].x, b[j].y);
            mma16<WE>(acc[j], lo.z, hi.z, lo.w, hi.w, b[j].z, b[j].w);
          }
        }
        // the block after next, or the next turn's
        if (kb + kAhead < KB)
          load_b(b, m0, kb + kAhead);
        else if (turn + 1 < turns)
          load_b(b, m0 + kStep, kb + kAhead - KB);
      }
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 8 * h + g;
      if (r >= count) continue;
      const float s = WE == kElemF16 && ad >= 0 ? unscale[r] : 1.0f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int c = m0 + Pc::column(k, t), n = a.M - c;  // columns there are
        float y[Pc::kCols] = {};
        if (a.y && a.y_vec && n >= Pc::kCols)
          read_y<YE>(mine + (turn & 1) * E::kYBytes + (h * kPer + k) * 512, y);
        else if (a.y)
          load_y<YE>(a.y + rows[r] * a.y_row + int64_t(c) * YS, n, y);
#pragma unroll
        for (int q = 0; q < Pc::kCols; ++q) {
          const int e = k * Pc::kCols + q;
          const float d = acc[e >> 1][2 * h + (e & 1)];
          if (ad >= 0) y[q] = WE == kElemF16 ? __fmaf_rn(d, s, y[q]) : __fadd_rn(d, y[q]);
        }
        store_y<YE>(a.out + rows[r] * a.out_row + int64_t(c) * YS, n, a.y_vec, y);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------ host --

// CTAs of a cluster, among which K is split: up to 8, while there are fewer than
// `limit` of them all and each has one of `pieces` pieces of K at least
int splits_of(int64_t clusters, int64_t limit, int64_t pieces) {
  int n = 1;
  while (n < 8 && clusters * n < limit && 2 * n <= pieces) n *= 2;
  return n;
}

LoraPlan plan_of(int64_t T, int64_t n, int64_t rank, int64_t K) {
  LoraPlan p{};
  const int64_t groups = std::min(n + 1, T);
  p.grouped = T > kLeaders;
  // a tile of 64 pays where an adapter fills it, by the mean, and there is work
  // enough for its preparation (4096 x 4096: 1024 tokens at rank 32 27 us with tiles
  // of 16, 30 with 64; 2048 tokens at rank 16 27 and 32, at rank 32 51 and 44)
  p.tm = T > 512 && T * rank > 32768 && T >= 32 * groups ? 64 : 16;
  p.tiles = int(p.grouped ? T / p.tm + groups : T);
  // about as many tiles have work; in tiles of 16 a warp has four blocks of 32 k at
  // least, or one where clusters are few
  p.busy = p.grouped ? T / p.tm + groups / 2 : (T + 15) / 16 + std::min(n, T) / 2;
  if (p.tm == 16) {
    const int64_t clusters = p.busy * (rank <= 16 ? 1 : (rank + 31) / 32);
    p.splits = splits_of(clusters, 304, K / 32 / (clusters < 32 ? 4 : 16));
  }
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  p.bytes = up(size_t(T) * size_t(rank) * 4);
  if (p.grouped) {
    p.sorted_off = p.bytes;
    p.tiles_off = p.sorted_off + up(size_t(T) * 4);
    p.n_off = p.tiles_off + up(size_t(p.tiles) * sizeof(LoraTile));
    p.bytes = p.n_off + 256;
  }
  return p;
}

// chunks of ranks side by side in the grid: they read the same x
template <int XE, int WE, int NT>
cudaError_t shrink16_nt(const LoraArgs &a, const LoraWork &w, const LoraPlan &p, cudaStream_t s) {
  const dim3 grid(unsigned(p.splits * ((a.rank + 8 * NT - 1) / (8 * NT))), unsigned(p.tiles));
  return launch_ex(k_lora_shrink16<XE, WE, NT>, grid, kShrinkThreads, 0, p.splits, p.grouped, s, a, w, p.splits);
}
template <int XE, int WE>
cudaError_t shrink16(const LoraArgs &a, const LoraWork &w, const LoraPlan &p, cudaStream_t s) {
  return a.rank <= 16 ? shrink16_nt<XE, WE, 2>(a, w, p, s) : shrink16_nt<XE, WE, 4>(a, w, p, s);
}
template <int XE, int WE, int NT>
cudaError_t shrink64_nt(const LoraArgs &a, const LoraWork &w, const LoraPlan &p, cudaStream_t s) {
  const dim3 grid(unsigned(p.splits * ((a.rank + 8 * NT - 1) / (8 * NT))), unsigned(p.tiles));
  return launch_ex(k_lora_shrink64<XE, WE, NT>, grid, kShrinkThreads, Ring<XE, NT>::kBytes, p.splits, true, s, a, w, p.splits);
}
template <int XE, int WE>
cudaError_t shrink64(const LoraArgs &a, const LoraWork &w, LoraPlan p, cudaStream_t s) {
  if constexpr (XE != kElemF32 || WE == kElemBF16)
    if (XE == kElemF32 || a.rank > 64) {
      p.splits = splits_of(p.busy, 160, a.K / 256);  // an SM has two CTAs, each four stages of 64 k at least
      return launch_lora_shrink_tc(XE, WE, a, w, p, s);
    }
  p.splits = splits_of(p.busy * ((a.rank + 63) / 64), 304, a.K / 256);
  if constexpr (XE != kElemF32 || WE != kElemBF16) {
    if (a.rank <= 16) return shrink64_nt<XE, WE, 2>(a, w, p, s);
    return a.rank <= 32 ? shrink64_nt<XE, WE, 4>(a, w, p, s) : shrink64_nt<XE, WE, 8>(a, w, p, s);
  }
  return cudaErrorInvalidValue;  // not reached
}

template <int WE, int YE>
cudaError_t expand16(const LoraArgs &a, const LoraWork &w, const LoraPlan &p, int sms, cudaStream_t s) {
  const int64_t groups = (a.M + 255) / 256;
  int turns = 1;  // of a CTA: several where enough CTAs remain
  while (turns < 8 && groups * p.tiles / (2 * turns) >= int64_t(sms) * 8) turns *= 2;
  const dim3 grid(unsigned((groups + turns - 1) / turns), unsigned(p.tiles));
  if (a.rank <= 32) return launch_ex(k_lora_expand<WE, YE, 1>, grid, kExpandThreads, Expand<WE, YE, 1>::kBytes, 1, true, s, a, w, turns);
  if (a.rank <= 64) return launch_ex(k_lora_expand<WE, YE, 2>, grid, kExpandThreads, Expand<WE, YE, 2>::kBytes, 1, true, s, a, w, turns);
  return launch_ex(k_lora_expand<WE, YE, 4>, grid, kExpandThreads, Expand<WE, YE, 4>::kBytes, 1, true, s, a, w, turns);
}

template <int WE, int TM>
cudaError_t run(int x_elem, int y_elem, const LoraArgs &a, const LoraWork &w, const LoraPlan &p, int sms, cudaStream_t s) {
  if (p.grouped) {
    const cudaError_t e = launch_ex(k_lora_group<TM>, dim3(1), kGroupThreads, 0, 1, false, s, a, w);
    if (e != cudaSuccess) return e;
  }
  if constexpr (TM == 64) {
    const cudaError_t e = x_elem == kElemF32 ? shrink64<kElemF32, WE>(a, w, p, s) : shrink64<WE, WE>(a, w, p, s);
    return e == cudaSuccess ? launch_lora_expand_tc(WE, y_elem, a, w, p, sms, s) : e;
  } else {
    const cudaError_t e = x_elem == kElemF32 ? shrink16<kElemF32, WE>(a, w, p, s) : shrink16<WE, WE>(a, w, p, s);
    if (e != cudaSuccess) return e;
    return y_elem == kElemF32 ? expand16<WE, kElemF32>(a, w, p, sms, s) : expand16<WE, WE>(a, w, p, sms, s);
  }
}

}  // namespace

size_t lora_workspace_bytes(int64_t n_tokens, int64_t n_adapters, int64_t rank, int64_t K, int64_t) {
  return plan_of(n_tokens, n_adapters, rank, K).bytes;
}

cudaError_t launch_lora(int x_elem, int w_elem, int y_elem, LoraArgs a, void *ws, cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  a.err = di->err_word;
  const LoraPlan p = plan_of(a.n_tokens, a.n_adapters, a.rank, a.K);
  uint8_t *base = static_cast<uint8_t *>(ws);
  LoraWork w{reinterpret_cast<float *>(base), nullptr, nullptr, nullptr};
  if (p.grouped) {
    w.sorted = reinterpret_cast<int32_t *>(base + p.sorted_off);
    w.tiles = reinterpret_cast<LoraTile *>(base + p.tiles_off);
    w.n_tiles = reinterpret_cast<int32_t *>(base + p.n_off);
  }
  const int sms = di->sm_count;
  if (w_elem == kElemBF16)
    return p.tm == 64 ? run<kElemBF16, 64>(x_elem, y_elem, a, w, p, sms, stream) : run<kElemBF16, 16>(x_elem, y_elem, a, w, p, sms, stream);
  return p.tm == 64 ? run<kElemF16, 64>(x_elem, y_elem, a, w, p, sms, stream) : run<kElemF16, 16>(x_elem, y_elem, a, w, p, sms, stream);
}

}  // namespace bq

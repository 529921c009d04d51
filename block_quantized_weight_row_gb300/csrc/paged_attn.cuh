// paged_attn.cuh — attention of few query rows per kv head over a paged,
// block-quantized KV cache (decode steps, drafted tokens): the streaming
// kernel. A quantized V cache is read by flash attention ("05. llama.cpp：从
// GGUF 文件到本地推理服务", §KV Cache 类型与 Flash Attention; the pages give no
// formula): s_ij = scale q_i . k^_j over the tokens that row i sees, o_i =
// sum_j softmax_j(s_i) v^_j, k^ and v^ being scale * code.
//
// Bound by reading the cache (0.56 or 1.06 bytes per value, each used once per
// query row): at the measured copy rate an SM has ~6 cycles per 4-bit token
// and kv head of 128 channels, so what counts is instructions per code.
//   - Products run on m16n8k16 binary16 matrix instructions with the query
//     rows as the 8 columns: K (tokens x channels) and V^T (channels x tokens)
//     are the 16-row operand, and their fragments are cut straight out of the
//     code words. A 4-bit code u in the low bits of a half-word IS the
//     binary16 subnormal u * 2^-24, exactly, so a word of 8 codes becomes four
//     operand registers with one mask each and one shift; codes in bits 4-7
//     read as 16 u, and the matching half of q is divided by 16 (exactly). The
//     products' adder aligns a subnormal by its nominal exponent, which costs
//     their sum up to 2^-17 (measured: 6e-6 of the output): nothing beside a
//     16-bit output's rounding, but fp32 calls turn the codes into u - 8 as
//     normal numbers (one more instruction per pair; 3e-7).
//   - The block scales stay out of the operands: a K block's two products
//     leave sum(q u) 2^-24, the accumulators start at -8 sum(q) 2^-24, and
//     d_k multiplies in fp32; d_v multiplies the weights in fp32, before their
//     one rounding to binary16. So codes and scales enter exactly. q is
//     brought to [2^10, 2^11) by a power of two per row (binary16 then holds
//     bf16 and fp16 q exactly); fp32 q and weights are split in two binary16
//     terms (22 bits), 2^-22 instead of 2^-11. A 16-bit output's weights take
//     one term: 2^-11 each, an eighth of bf16's own rounding.
//   - Weights d_v p are scaled by a power of two per warp that keeps them
//     in binary16 whatever the V scales are, and a row's maximum is only raised
//     (and the accumulators rescaled) when a score passes it by 2^8 (16-bit
//     calls; d_v below 2^6) or 2 (fp32 calls; d_v in [2^13, 2^14)): with fp32
//     accumulators any common factor serves. The terms end at binary16's
//     smallest subnormal: d_v p is off by up to 2^-25, that is 2^-29 (16-bit) or
//     2^-37 (fp32) of the warp's largest d_v and the row's largest p there. The
//     headroom of the 16-bit calls would cost an fp32 call with 131071 tokens
//     beside dominant ones up to 2^-12 of its output; so 2^-20.
//   - Softmax statistics and the accumulators are fp32; transposing the
//     weights from "row = token" to "column = query row" is one movmatrix.
//   - A warp streams its own tiles through a private ring of asynchronous
//     16-byte copies; warps of a CTA meet only where a segment ends.
// Work: the tiles of all (sequence, kv head, row group) segments form one
// sequence that is cut into equal pieces, one per CTA, on the device (lengths
// stay there), so ragged batches load every SM alike. A segment inside a piece
// is finished there; one that is cut leaves partial results for the combine
// launch, which merges them in a fixed order.
// Measured (8 kv heads of 128 channels, bf16): 64 ragged sequences of up to
// 8192 tokens, 32 query heads, 4 bits, 100.5 us, 3.1 TB/s of cache (132 us in
// fp32); 4 sequences of up to 131071 tokens, 16 query heads, 8-bit V, 101 us, 4.9
// TB/s (0.73 of the copy rate); one of 777 tokens in fp32 12.3 us. With the products and the softmax
// taken out (copies, segment starts and combine left) the first takes 63 us,
// the second 81: what is above that is instruction issue (452 per 16 tokens
// and warp, ALU pipe 48% busy), and the pieces' unequal ends (67 to 95 us).
#pragma once

#include "bq_device.cuh"
#include "bq_internal.h"
#include "paged_attn.h"

namespace bq {
namespace paged {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kRaise = 8.0f;   // a maximum is raised when passed by this much (base-2 units; fp32 calls: below)
constexpr float kNoMax = -3.402823466e38f;  // no score seen yet
constexpr int kNoExp = 0x7fffffff;  // no V scale seen yet
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a b + (c0, c1, c0, c1)
__device__ __forceinline__ void mma16816_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1, float c0, float c1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 half2_floats(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Two 4-bit codes (bits 0-3 and 16-19 of w, or with _hi bits 4-7 and 20-23)
// as binary16 u - 8, exactly: 1024 + u - 1032, (1024 + 16 u) / 16 - 72.
__device__ __forceinline__ uint32_t codes4_lo(uint32_t w) { return hsub2((w & 0x000f000fu) | 0x64006400u, 0x64086408u); }
__device__ __forceinline__ uint32_t codes4_hi(uint32_t w) { return hfma2((w & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, 0xd480d480u); }

// Token of fragment row slot r (0..7; slot r + 8 is 8 tokens on). Any
// bijection serves (weights and V rows use the same one); this one lets the
// eight lanes of a shared-memory phase read K rows of both parities, and a
// V load's four lanes consecutive rows: no bank conflicts.
__device__ __forceinline__ int slot_token(int r) { return (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1; }

// Shared-memory chunk (16 bytes) of chunk c of token t's codes, C chunks per row
template <int C>
__device__ __forceinline__ int swz_k(int t, int c) {
  if constexpr (C == 8) return c ^ (t & 1);
  if constexpr (C == 16) return c ^ (c >> 3) ^ ((t & 1) << 1);
  return c;
}
template <int C>
__device__ __forceinline__ int swz_v(int t, int c) {
  if constexpr (C == 4) return c ^ (t & 2);
  if constexpr (C == 8) return c ^ ((t & 3) << 1);
  if constexpr (C == 16) return c ^ (((t & 1) << 2) | ((t & 2) >> 1));
  return c;
}

// N bytes at byte `at` of token t's row, from a swizzled tile
template <int N, int C, bool IS_V>
__device__ __forceinline__ void lds_piece(const uint8_t *tile, int t, int at, uint32_t (&w)[(N + 3) / 4]) {
  auto addr = [&](int o) {
    const int c = o >> 4;
    return tile + t * (C * 16) + ((IS_V ? swz_v<C>(t, c) : swz_k<C>(t, c)) << 4) + (o & 15);
  };
  if constexpr (N % 16 == 0) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      const uint4 v = *reinterpret_cast<const uint4 *>(addr(at + 16 * i));
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const uint2 v = *reinterpret_cast<const uint2 *>(addr(at + 8 * i));
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    }
  } else if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = *reinterpret_cast<const uint32_t *>(addr(at + 4 * i));
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t h = *reinterpret_cast<const uint16_t *>(addr(at + 2 * i));
      w[i / 2] = (i & 1) ? w[i / 2] | (h << 16) : h;
    }
  }
}

// The NB binary16 scales of token t (row of the tile)
template <int NB>
__device__ __forceinline__ void lds_scales(const uint8_t *tile, int t, uint32_t (&w)[(NB + 1) / 2]) {
  const uint8_t *p = tile + t * NB * 2;
  if constexpr (NB % 8 == 0) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (NB % 4 == 0) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x, w[1] = v.y;
  } else if constexpr (NB % 2 == 0) {
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint32_t h = reinterpret_cast<const uint16_t *>(p)[i];
      w[i / 2] = (i & 1) ? w[i / 2] | (h << 16) : h;
    }
  }
}
template <int N>
__device__ __forceinline__ float scale_of(const uint32_t (&w)[N], int b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[b / 2]));
  return (b & 1) ? f.y : f.x;
}

// bytes: 16, or 0 to fill with zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Sizes of one instantiation. R: groups of 8 query rows per pass; TERMS:
// binary16 terms of q and the weights.
template <int NB, int KT, int VT, int R, int TERMS>
struct Cfg {
  static constexpr int D = NB * 32;
  static constexpr int RBK = NB * Codes<KT>::kBytes, RBV = NB * Codes<VT>::kBytes;
  static constexpr int SUB = 16 * (RBK + RBV) + 2 * 16 * NB * 2;   // bytes of 16 tokens
  static constexpr int kHalf = 112 * 1024;                          // two CTAs per SM
  static constexpr int TT = 2 * 2 * SUB * kWarps <= kHalf ? 2 : 1;  // 16-token tiles per stage
  static constexpr int STAGE = TT * SUB;
  static constexpr bool kTwo = 2 * STAGE * kWarps <= kHalf;
  static constexpr int S = 3 * STAGE * kWarps <= kHalf ? 3 : kTwo ? 2 : 3;  // ring stages
  static constexpr int TOK = 16 * TT;                               // tokens per stage
  static constexpr int ROWS = 8 * R;
  static constexpr int OP = D + 8;                                  // pitch of a merge row (floats)
  static constexpr int kRing = kWarps * S * STAGE;
  static constexpr int kMerge = kWarps * ROWS * OP * 4 + kWarps * ROWS * 8;
  static constexpr int QV = NB == 3 ? 4 : NB;                       // channels per lane while q is prepared
  static constexpr int QP = TERMS * D * 2 + 64;                     // pitch of a prepared q row (bytes)
  static constexpr int kOffQ = kRing > kMerge ? kRing : kMerge;
  static constexpr int kOffScale = kOffQ + ROWS * QP;               // [row]: score factor
  static constexpr int kOffInit = kOffScale + ROWS * 4;             // [row][block]: what the products start at
  static constexpr int kSmem = kOffInit + ROWS * NB * 4;
  static constexpr int kCtas = kTwo && 2 * (kSmem + 1024) <= 227 * 1024 && NB * R <= 4 ? 2 : 1;
};

// Tiles of a sequence: [t_lo, t_lo + tiles) of `tok` tokens hold every token
// that any of its rows sees; a sequence with rows has at least one tile, so
// that its output is written even when no row sees a token.
// `cost` counts a segment's start and merge too, in tiles: a batch's short
// sequences would otherwise leave their CTAs far behind the others (512
// tokens' worth: a ragged decode batch of 64 sequences took 114 us without,
// 107 with 256, 101 with 512, 102 with 768).
constexpr int kSegTokens = 512;
struct SeqTiles {
  int t_lo, tiles, cost, groups;  // per (kv head, row group)
};
__device__ __forceinline__ SeqTiles seq_tiles(const PagedAttnArgs &a, const SeqSpan &s, int tok, int rows) {
  SeqTiles t{0, 0, 0, 0};
  const int n_rows = s.q_len * a.group;
  if (s.q_len == 0 || n_rows > a.tc_rows) return t;
  int lo, hi, lo1, hi1;
  seen_range(s, 0, a.causal, a.window, lo, hi1);
  seen_range(s, s.q_len - 1, a.causal, a.window, lo1, hi);
  t.t_lo = lo / tok;
  const int t_hi = (hi + tok - 1) / tok;
  t.tiles = t_hi > t.t_lo ? t_hi - t.t_lo : 1;
  t.cost = t.tiles + kSegTokens / tok;
  t.groups = (n_rows + rows - 1) / rows;
  return t;
}

__device__ __forceinline__ SeqSpan load_span(const PagedAttnArgs &a, int b, bool report) {
  bool bad;
  const int64_t most = min(int64_t(a.max_kv), int64_t(a.max_pages) * a.sh.page_size);
  const SeqSpan s = checked_span(__ldg(a.q_start + b), __ldg(a.q_start + b + 1), __ldg(a.kv_len + b), a.n_q, most, bad);
  if (bad && report) atomicOr(a.err, kErrIndex);
  return s;
}

template <int ELEM>
__device__ __forceinline__ void store_out4(uint8_t *p, float4 v) {
  if constexpr (ELEM == kElemF32)
    *reinterpret_cast<float4 *>(p) = v;
  else
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_pair<ELEM>(v.x, v.y), pack_pair<ELEM>(v.z, v.w));
}
__device__ __forceinline__ void store_out4(int elem, uint8_t *row, int ch, float4 v) {
  if (elem == kElemF32)
    store_out4<kElemF32>(row + ch * 4, v);
  else if (elem == kElemF16)
    store_out4<kElemF16>(row + ch * 2, v);
  else
    store_out4<kElemBF16>(row + ch * 2, v);
}

// V consecutive q values from channel ch, as fp32
template <int V>
__device__ __forceinline__ void load_q(int elem, const uint8_t *row, int ch, float (&x)[V]) {
  if (elem == kElemF32) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 v = __ldg(reinterpret_cast<const float2 *>(row + (ch + i) * 4));
      x[i] = v.x, x[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(row + (ch + i) * 2));
      const float2 v = elem == kElemF16 ? unpack_pair<kElemF16>(w) : unpack_pair<kElemBF16>(w);
      x[i] = v.x, x[i + 1] = v.y;
    }
  }
}

template <int NB, int KT, int VT, int R, int TERMS>
__global__ void __launch_bounds__(kThreads, (Cfg<NB, KT, VT, R, TERMS>::kCtas))
    k_paged_stream(const __grid_constant__ PagedAttnArgs a, int min_tiles) {
  using C = Cfg<NB, KT, VT, R, TERMS>;
  constexpr int D = C::D, TT = C::TT, S = C::S, TOK = C::TOK, ROWS = C::ROWS, OP = C::OP;
  constexpr int CK = C::RBK / 16, CV = C::RBV / 16;            // 16-byte chunks per row
  constexpr int UK = C::RBK / kUnitsK, UV = C::RBV / kUnitsV;  // bytes of a lane's piece of a row
  constexpr bool K4 = KT == kTypeQ4_0, V4 = VT == kTypeQ4_0;
  // 4-bit codes as subnormals u * 2^-24 (16-bit calls), and then the factor
  // of the products' accumulators
  constexpr bool KSUB = K4 && TERMS == 1, VSUB = V4 && TERMS == 1;
  constexpr float kKUnit = KSUB ? 16777216.0f : 1.0f, kVUnit = VSUB ? 16777216.0f : 1.0f;
  // A maximum is raised when passed by kPass, the largest V scale brought to
  // [2^kHeadV, 2^(kHeadV + 1)): weights stay below 2^14 or 2^15. (64 ragged
  // sequences of up to 8192 tokens in fp32: 132 us; 137 raised by anything, 136
  // with the 16-bit calls' 2^8.)
  constexpr float kPass = TERMS == 1 ? kRaise : 1.0f;
  constexpr int kHeadV = TERMS == 1 ? 5 : 13;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t sh_scan[kWarps + 1];
  __shared__ int64_t sh_find[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  pdl_launch_dependents();  // the combine may become resident; it waits for this grid

  // ---- this CTA's piece [t0, t1) of all tiles ----
  const int per_thread = (a.n_seqs + kThreads - 1) / kThreads;
  const int b_first = min(int(threadIdx.x) * per_thread, a.n_seqs), b_last = min(b_first + per_thread, a.n_seqs);
  int64_t mine = 0;
  for (int b = b_first; b < b_last; ++b) {
    const SeqTiles t = seq_tiles(a, load_span(a, b, blockIdx.x == 0), TOK, ROWS);
    mine += int64_t(t.cost) * t.groups * a.sh.n_kv;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh_scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh_scan[w];
    total += sh_scan[w];
  }
  const int64_t piece = max((total + gridDim.x - 1) / gridDim.x, int64_t(min_tiles));
  const int64_t t0 = min(piece * blockIdx.x, total), t1 = min(t0 + piece, total);
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, -1);
  if (t0 >= t1) {
    pdl_wait();
    return;
  }
  if (before <= t0 && t0 < before + mine) {
    int64_t at = before;
    for (int b = b_first; b < b_last; ++b) {
      const SeqTiles t = seq_tiles(a, load_span(a, b, false), TOK, ROWS);
      const int64_t n = int64_t(t.cost) * t.groups * a.sh.n_kv;
      if (t0 < at + n) {
        sh_find[0] = b;
        sh_find[1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  int seq = int(sh_find[0]);
  int64_t seq_at = sh_find[1];  // first tile of the sequence

  uint8_t *ring = smem + warp * S * C::STAGE;
  const uint32_t ring_u = smem_u32(ring);
  // where this lane's 16-byte chunks of a 16-token tile go
  uint32_t dst_k[(16 * CK + 31) / 32], dst_v[(16 * CV + 31) / 32];
#pragma unroll
  for (int i = 0; i < (16 * CK + 31) / 32; ++i) {
    const int q = lane + 32 * i;
    dst_k[i] = uint32_t(q / CK * C::RBK + (swz_k<CK>(q / CK, q % CK) << 4));
  }
#pragma unroll
  for (int i = 0; i < (16 * CV + 31) / 32; ++i) {
    const int q = lane + 32 * i;
    dst_v[i] = uint32_t(16 * C::RBK + q / CV * C::RBV + (swz_v<CV>(q / CV, q % CV) << 4));
  }
  const bool scales_v = lane >= 2 * NB;
  const uint32_t dst_s = 16 * (C::RBK + C::RBV) + lane * 16;
  const int64_t scale_at = (scales_v ? a.vp.scale_off : a.kp.scale_off) + (scales_v ? lane - 2 * NB : lane) * 16;
  float *merge_o = reinterpret_cast<float *>(smem);
  float2 *merge_ml = reinterpret_cast<float2 *>(smem + kWarps * ROWS * OP * 4);
  uint8_t *q_rows = smem + C::kOffQ;
  float *q_scale = reinterpret_cast<float *>(smem + C::kOffScale), *q_init = reinterpret_cast<float *>(smem + C::kOffInit);

  for (int64_t at = t0; at < t1;) {
    // ---- the segment that holds tile `at` ----
    SeqSpan span = load_span(a, seq, false);
    SeqTiles st = seq_tiles(a, span, TOK, ROWS);
    while (at >= seq_at + int64_t(st.cost) * st.groups * a.sh.n_kv) {
      seq_at += int64_t(st.cost) * st.groups * a.sh.n_kv;
      span = load_span(a, ++seq, false);
      st = seq_tiles(a, span, TOK, ROWS);
    }
    const int64_t seg = (at - seq_at) / st.cost, seg_at = seq_at + seg * st.cost, seg_end = seg_at + st.cost;
    const int kvh = int(seg / st.groups), rg = int(seg - int64_t(kvh) * st.groups);
    const int64_t stop = min(seg_end, t1);
    const int n_rows = span.q_len * a.group, row0 = rg * ROWS, rows = min(ROWS, n_rows - row0);
    // tokens that some row of the group sees, and tokens that all of them see
    int lo_any, hi_any, lo_all, hi_all;
    seen_range(span, row0 / a.group, a.causal, a.window, lo_any, hi_all);
    seen_range(span, (row0 + rows - 1) / a.group, a.causal, a.window, lo_all, hi_any);
    // the segment's fixed cost comes before its tiles
    const int fixed = st.cost - st.tiles;
    int tile = st.t_lo + max(int(at - seg_at) - fixed, 0), tile_end = st.t_lo + max(int(stop - seg_at) - fixed, 0);
    tile = max(tile, lo_any / TOK);
    tile_end = min(tile_end, (hi_any + TOK - 1) / TOK);

    // ---- the warp's first tiles are on their way while q is prepared ----
    const int64_t head_k = a.kp.head_bytes, head_v = a.vp.head_bytes;
    const int32_t *table = a.page_table + int64_t(seq) * a.table_stride;
    const uint8_t *kh = a.kp.base + int64_t(kvh) * head_k, *vh = a.vp.base + int64_t(kvh) * head_v;
    const int64_t page_k = head_k * a.sh.n_kv, page_v = head_v * a.sh.n_kv;
    // A stage: 16-token tiles, each within one page. A tile outside what any row
    // sees (its table entry may be stale: before a window too), or on a page
    // outside the pool (never read: reported), is zero-filled with the pool's
    // first tile as the address.
    auto issue = [&](int ti, int stage) {
      if (ti < tile_end) {
#pragma unroll
        for (int u = 0; u < TT; ++u) {
          const int tok = ti * TOK + u * 16;
          const bool seen = tok < hi_any && tok + 16 > lo_any;
          const int pi = token_page(a.sh, tok);
          uint32_t page = seen ? uint32_t(__ldg(table + pi)) : 0u;
          uint32_t place = uint32_t(tok - pi * a.sh.page_size), bytes = seen ? 16u : 0u;
          if (page >= uint64_t(a.sh.n_pages)) {
            if (lane == 0) atomicOr(a.err, kErrIndex);
            page = place = bytes = 0u;
          }
          const uint8_t *tk = kh + int64_t(page) * page_k, *tv = vh + int64_t(page) * page_v;
          const uint32_t base = ring_u + stage * C::STAGE + u * C::SUB;
          const uint8_t *sk = tk + place * C::RBK + lane * 16, *sv = tv + place * C::RBV + lane * 16;
#pragma unroll
          for (int i = 0; i < (16 * CK + 31) / 32; ++i)
            if (16 * CK % 32 == 0 || lane + 32 * i < 16 * CK) cp_async16(base + dst_k[i], sk + i * 512, bytes);
#pragma unroll
          for (int i = 0; i < (16 * CV + 31) / 32; ++i)
            if (16 * CV % 32 == 0 || lane + 32 * i < 16 * CV) cp_async16(base + dst_v[i], sv + i * 512, bytes);
          // scales: 2 NB chunks of K's, then as many of V's
          if (lane < 4 * NB) cp_async16(base + dst_s, (scales_v ? tv : tk) + (place * NB * 2 + scale_at), bytes);
        }
      }
      cp_commit();
    };
    int ti = tile + warp;
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(ti + s * kWarps, s);

    // ---- this lane's columns: rows 2c, 2c + 1 of each group of 8 ----
    int lo[R][2], hi[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = min(row0 + 8 * r + 2 * c + e, n_rows - 1);
        seen_range(span, row / a.group, a.causal, a.window, lo[r][e], hi[r][e]);
      }
    // q as operand columns, a warp per row (every warp for itself would cost a
    // segment as much as 400 of its tokens): scaled, split, and stored as
    // [block][unit][fragment pair] so that a lane (row, unit) reads 16 bytes
    // per block
#pragma unroll
    for (int r = 0; r < R; ++r) {
      constexpr int V = C::QV;
      const int local = 8 * r + warp, row = row0 + local, ch = lane * V;
      float x[V];
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = 0.0f;
      if (row < n_rows && ch < D) {
        const int tok = row / a.group, head = kvh * a.group + (row - tok * a.group);
        load_q<V>(a.elem, a.q + int64_t(span.q0 + tok) * a.q_token + int64_t(head) * a.q_head, ch, x);
      }
      if constexpr (NB != 3) {
        if (a.rotate) {  // spans 1, 2, ..., 32 in order: below V in the lane, then across
#pragma unroll
          for (int w = 1; w < V; w <<= 1)
#pragma unroll
            for (int i = 0; i < V; ++i)
              if ((i & w) == 0) {
                const float p = x[i], q = x[i + w];
                x[i] = __fadd_rn(p, q);
                x[i + w] = __fsub_rn(p, q);
              }
#pragma unroll
          for (int w = 1; w < 64 / V; w <<= 1)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float q = __shfl_xor_sync(kFull, x[i], w);
              x[i] = (lane & w) ? __fsub_rn(q, x[i]) : __fadd_rn(x[i], q);
            }
#pragma unroll
          for (int i = 0; i < V; ++i) x[i] = __fmul_rn(x[i], 0.125f);
        }
      }
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
      for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, w));
      // 2^k brings the row's largest value to [2^10, 2^11)
      const int k = top > 0.0f ? min(10 + 127 - int(__float_as_uint(top) >> 23), 110) : 0;
      // (the scale's sign goes into q). The factor stays positive, also for a
      // scale of 0 or a product below binary32's range: it multiplies the -infinity
      // of masked scores and divides; any score is below 2^42 times it, ~0.
      const float up = copysignf(__int_as_float((127 + k) << 23), a.scale_log2);
      if (lane == 0) q_scale[local] = fmaxf(fabsf(a.scale_log2) * kKUnit * __int_as_float((127 - k) << 23), 1e-37f);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // position of the channel: 4-bit codes (c, c + 2) of a unit's low
        // channels, of its high ones (read as 16 u: q / 16), then (c + 1, c + 3)
        const int e = (ch + i) & 31;
        const int unit = K4 ? (e & 15) >> 2 : e >> 3, high = K4 ? e >> 4 : 0;
        const int half = K4 ? (e & 1) * 4 + high * 2 + ((e >> 1) & 1) : e & 7;
        float y = x[i] * up;
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          const __half z = __float2half_rn(y);
          const float f = __half2float(z);
          if (ch < D)
            *reinterpret_cast<__half *>(q_rows + local * C::QP + t * D * 2 + ((ch + i) >> 5) * 64 + unit * 16 + half * 2) =
                KSUB && high ? __float2half_rn(f * 0.0625f) : z;
          sum += f;
          y -= f;
        }
      }
      if constexpr (KSUB) {  // the products start at -8 sum(q) of the block
#pragma unroll
        for (int w = 1; w < 32 / V; w <<= 1) sum += __shfl_xor_sync(kFull, sum, w);
        if (lane % (32 / V) == 0 && ch < D) q_init[local * NB + (ch >> 5)] = sum * (-8.0f / kKUnit);
      }
    }
    __syncthreads();
    uint32_t qf[R][TERMS][NB][4];
    float init[R][NB][2], qscale[R][2];  // score = qscale * sum_b d_k[b] * product[b]
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint4 v = *reinterpret_cast<const uint4 *>(q_rows + (8 * r + g) * C::QP + t * D * 2 + b * 64 + c * 16);
          qf[r][t][b][0] = v.x, qf[r][t][b][1] = v.y, qf[r][t][b][2] = v.z, qf[r][t][b][3] = v.w;
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qscale[r][e] = q_scale[8 * r + 2 * c + e];
#pragma unroll
        for (int b = 0; b < NB; ++b) init[r][b][e] = KSUB ? q_init[(8 * r + 2 * c + e) * NB + b] : 0.0f;
      }
    }

    float m[R][2], l[R][2], limit[R][2], o[R][NB][2][4];  // limit: the unscaled score that raises m
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r][0] = m[r][1] = kNoMax;
      limit[r][0] = limit[r][1] = kNoMax;
      l[r][0] = l[r][1] = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[r][b][i >> 2][i & 3] = 0.0f;
    }
    int vexp = kNoExp;  // weights are multiplied by 2^vexp

    // ---- the tiles ----
    int stage = 0;
    for (; ti < tile_end; ti += kWarps) {
      issue(ti + (S - 1) * kWarps, stage == 0 ? S - 1 : stage - 1);
      cp_wait<S - 1>();
      __syncwarp();
      const uint8_t *buf = ring + stage * C::STAGE;
      const bool full = ti * TOK >= lo_all && (ti + 1) * TOK <= hi_all;

      float s[TT][R][4];
#pragma unroll
      for (int u = 0; u < TT; ++u) {
        const uint8_t *sub = buf + u * C::SUB;
        uint32_t kw[2][UK / 4], ks[2][(NB + 1) / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = slot_token(g) + 8 * h;
          lds_piece<UK, CK, false>(sub, t, c * UK, kw[h]);
          lds_scales<NB>(sub + 16 * (C::RBK + C::RBV), t, ks[h]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) s[u][r][0] = s[u][r][1] = s[u][r][2] = s[u][r][3] = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t A[2][4];  // [token half][fragment pair], as qf
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (K4) {
              const uint32_t w = kw[h][b], v = w >> 8;
              A[h][0] = KSUB ? w & 0x000f000fu : codes4_lo(w);
              A[h][1] = KSUB ? w & 0x00f000f0u : codes4_hi(w);
              A[h][2] = KSUB ? v & 0x000f000fu : codes4_lo(v);
              A[h][3] = KSUB ? v & 0x00f000f0u : codes4_hi(v);
            } else {
              const uint2 p = codes_to_f16x2(kw[h][2 * b]), q = codes_to_f16x2(kw[h][2 * b + 1]);
              A[h][0] = p.x, A[h][1] = p.y, A[h][2] = q.x, A[h][3] = q.y;
            }
          }
          const float d0 = scale_of(ks[0], b), d1 = scale_of(ks[1], b);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float acc[4];
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t) {
              if (t == TERMS - 1)
                mma16816_from(acc, A[0][0], A[1][0], A[0][1], A[1][1], qf[r][t][b][0], qf[r][t][b][1], init[r][b][0], init[r][b][1]);
              else
                mma16816(acc, A[0][0], A[1][0], A[0][1], A[1][1], qf[r][t][b][0], qf[r][t][b][1]);
              mma16816(acc, A[0][2], A[1][2], A[0][3], A[1][3], qf[r][t][b][2], qf[r][t][b][3]);
            }
            s[u][r][0] = fmaf(d0, acc[0], s[u][r][0]);
            s[u][r][1] = fmaf(d0, acc[1], s[u][r][1]);
            s[u][r][2] = fmaf(d1, acc[2], s[u][r][2]);
            s[u][r][3] = fmaf(d1, acc[3], s[u][r][3]);
          }
        }
      }
      // V scales of the lane's two tokens per 16; outside what any row sees
      // they count as zero, whatever the page holds there
      uint32_t vs[TT][2][(NB + 1) / 2];
      uint32_t vmax = 0;
#pragma unroll
      for (int u = 0; u < TT; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = slot_token(g) + 8 * h;
          lds_scales<NB>(buf + u * C::SUB + 16 * (C::RBK + C::RBV) + 16 * NB * 2, t, vs[u][h]);
          if (!full) {
            const int tok = ti * TOK + u * 16 + t;
            const bool live = tok >= lo_any && tok < hi_any;
#pragma unroll
            for (int i = 0; i < (NB + 1) / 2; ++i) vs[u][h][i] = live ? vs[u][h][i] : 0u;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (tok < lo[r][e] || tok >= hi[r][e]) s[u][r][2 * h + e] = -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < (NB + 1) / 2; ++i) vmax = max_u16x2(vmax, vs[u][h][i]);  // scales are not negative
        }
      // power of two that brings the largest V scale seen there: the binary16
      // exponent (subnormals count as the smallest normal) decides
      vmax = __reduce_max_sync(kFull, max(vmax & 0x7fffu, (vmax >> 16) & 0x7fffu));
      const int need = 15 + kHeadV - max(int(vmax >> 10), 1);  // 2^kHeadV / 2^(e - 15)
      if (need < vexp) {  // warp-uniform; rare after the first tile
        if (vexp != kNoExp) {
          const float f = __int_as_float((127 + need - vexp) << 23);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            l[r][0] *= f;
            l[r][1] *= f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int i = 0; i < 8; ++i) o[r][b][i >> 2][i & 3] *= f;
          }
        }
        vexp = need;
      }

      // ---- running maximum ----
      bool raise = false;
      float top[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(s[0][r][e], s[0][r][2 + e]);
#pragma unroll
          for (int u = 1; u < TT; ++u) t = fmaxf(t, fmaxf(s[u][r][e], s[u][r][2 + e]));
          top[r][e] = t;
          raise = raise || t > limit[r][e];
        }
      if (__any_sync(kFull, raise)) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = top[r][e];
            t = fmaxf(t, __shfl_xor_sync(kFull, t, 4));
            t = fmaxf(t, __shfl_xor_sync(kFull, t, 8));
            t = fmaxf(t, __shfl_xor_sync(kFull, t, 16));
            // a whole number, so that the weights' power of two joins it exactly
            const float mn = fmaxf(m[r][e], ceilf(t * qscale[r][e]));
            const float al = ex2(m[r][e] - mn);
            m[r][e] = mn;
            limit[r][e] = (mn + kPass) / qscale[r][e];
            l[r][e] *= al;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                o[r][b][mt][e] *= al;
                o[r][b][mt][2 + e] *= al;
              }
          }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float off[2] = {float(vexp) - m[r][0], float(vexp) - m[r][1]};
#pragma unroll
        for (int u = 0; u < TT; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = ex2(fmaf(s[u][r][i], qscale[r][i & 1], off[i & 1]));  // 0 for a masked score: the maximum is finite
            l[r][i & 1] += p;
            s[u][r][i] = p;
          }
      }

      // ---- weights times V ----
#pragma unroll
      for (int u = 0; u < TT; ++u) {
        const uint8_t *sub = buf + u * C::SUB + 16 * C::RBK;
        uint32_t vw[4][(UV + 3) / 4];  // fragment slots 2c, 2c + 1, 2c + 8, 2c + 9
        lds_piece<UV, CV, true>(sub, c, g * UV, vw[0]);
        lds_piece<UV, CV, true>(sub, 4 + (c ^ 1), g * UV, vw[1]);
        lds_piece<UV, CV, true>(sub, 8 + c, g * UV, vw[2]);
        lds_piece<UV, CV, true>(sub, 12 + (c ^ 1), g * UV, vw[3]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t A[2][4];  // two 16-channel tiles of the block
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if constexpr (V4) {
              // half-word b of both tokens of the pair side by side
              const uint32_t X = __byte_perm(vw[2 * k][b / 2], vw[2 * k + 1][b / 2], (b & 1) ? 0x7632 : 0x5410);
              const uint32_t Y = X >> 8;
              A[0][2 * k] = VSUB ? hsub2(X & 0x000f000fu, 0x00080008u) : codes4_lo(X);      // channels 2g
              A[0][2 * k + 1] = VSUB ? hsub2(Y & 0x000f000fu, 0x00080008u) : codes4_lo(Y);  // 2g + 1
              A[1][2 * k] = VSUB ? hsub2(X & 0x00f000f0u, 0x00800080u) : codes4_hi(X);      // 16 + 2g (subnormal: 16 u)
              A[1][2 * k + 1] = VSUB ? hsub2(Y & 0x00f000f0u, 0x00800080u) : codes4_hi(Y);
            } else {
              // bytes of both tokens interleaved, then the exact binary16 codes
              const uint32_t w0 = vw[2 * k][b], w1 = vw[2 * k + 1][b];
              const uint2 p = codes_to_f16x2(__byte_perm(w0, w1, 0x5140)), q = codes_to_f16x2(__byte_perm(w0, w1, 0x7362));
              A[0][2 * k] = p.x, A[0][2 * k + 1] = p.y;  // channels 4g, 4g + 1
              A[1][2 * k] = q.x, A[1][2 * k + 1] = q.y;  // 4g + 2, 4g + 3
            }
          }
          const float d0 = scale_of(vs[u][0], b), d1 = scale_of(vs[u][1], b);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float w0 = s[u][r][0] * d0, w1 = s[u][r][1] * d0, w2 = s[u][r][2] * d1, w3 = s[u][r][3] * d1;
            // The matrix instruction's adder truncates. One term: along the
            // cache that adds up to some 1e-5 of the output, nothing beside
            // 16 bits. Two: 16 tokens at a time, then a rounded addition.
            float fresh[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int t = 0; t < TERMS; ++t) {
              const uint32_t h0 = half2_bits(w0, w1), h1 = half2_bits(w2, w3);
              const uint32_t b0 = movmatrix_trans(h0), b1 = movmatrix_trans(h1);
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                float(&acc)[4] = TERMS == 1 ? o[r][b][mt] : fresh[mt];
                mma16816(acc, A[mt][0], A[mt][1], A[mt][2], A[mt][3], b0, b1);
              }
              if (t + 1 < TERMS) {
                const float2 f0 = half2_floats(h0), f1 = half2_floats(h1);
                w0 -= f0.x, w1 -= f0.y, w2 -= f1.x, w3 -= f1.y;
              }
            }
            if constexpr (TERMS > 1) {
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[r][b][mt][i] += fresh[mt][i];
            }
          }
        }
      }
      stage = stage + 1 == S ? 0 : stage + 1;
      __syncwarp();  // every lane has read the stage before it is refilled
    }
    cp_wait<0>();
    __syncthreads();  // the rings become the merge buffer

    // ---- merge the warps ----
    {
      const float down = vexp == kNoExp ? 0.0f : __int_as_float((127 - vexp) << 23) * kVUnit;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[r][e] += __shfl_xor_sync(kFull, l[r][e], 4);
          l[r][e] += __shfl_xor_sync(kFull, l[r][e], 8);
          l[r][e] += __shfl_xor_sync(kFull, l[r][e], 16);
          const int row = warp * ROWS + 8 * r + 2 * c + e;
          if (g == 0) merge_ml[row] = make_float2(m[r][e], l[r][e] * (vexp == kNoExp ? 0.0f : __int_as_float((127 - vexp) << 23)));
          float *dst = merge_o + row * OP;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              const float f = VSUB && mt ? down * 0.0625f : down;
              const int ch = b * 32 + (V4 ? 16 * mt + 2 * g : 4 * g + 2 * mt);
              *reinterpret_cast<float2 *>(dst + ch) = make_float2(o[r][b][mt][e] * f, o[r][b][mt][2 + e] * f);
            }
        }
      }
    }
    __syncthreads();
    const bool whole = seg_at >= t0 && seg_end <= t1;
    const int slot = seg_at >= t0 ? 1 : 0;  // partial results: 1 for a segment that starts in this piece
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), ch = (i - r * (D / 4)) * 4;
      float top = kNoMax;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, merge_ml[w * ROWS + r].x);
      float sum = 0.0f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = merge_ml[w * ROWS + r];
        if (ml.y == 0.0f) continue;  // the warp saw no token of this row
        const float f = ex2(ml.x - top);
        const float4 v = *reinterpret_cast<const float4 *>(merge_o + (w * ROWS + r) * OP + ch);
        sum = fmaf(ml.y, f, sum);
        acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y), acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
      }
      if (whole) {
        const int tok = (row0 + r) / a.group, head = kvh * a.group + (row0 + r - tok * a.group);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint8_t *row = a.o + int64_t(span.q0 + tok) * a.o_token + int64_t(head) * a.o_head;
        store_out4(a.elem, row, ch, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (ch == 0 && a.lse)
          a.lse[int64_t(span.q0 + tok) * a.n_heads + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
      } else {
        const int64_t p = (int64_t(blockIdx.x) * 2 + slot) * ROWS + r;
        *reinterpret_cast<float4 *>(a.part_o + p * D + ch) = acc;
        if (ch == 0) a.part_ml[p] = make_float2(top, sum);
      }
    }
    if (!whole && slot == 1 && threadIdx.x == 0)
      a.meta[blockIdx.x] = make_int4(seq, kvh, rg, int((seg_end - 1) / piece));
    at = stop;
    __syncthreads();  // the merge buffer becomes the rings again
  }
  // launched beside the many-row kernel of the same call (they share no
  // output): ends after it, so that what follows is ordered after both
  pdl_wait();
}

// Each head dimension's instantiations are a translation unit of their own.
template <int NB, int KT, int VT, int R, int TERMS>
cudaError_t launch_stream_one(const PagedAttnArgs &a, int grid, int min_tiles, bool beside, cudaStream_t stream) {
  using C = Cfg<NB, KT, VT, R, TERMS>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void *>(k_paged_stream<NB, KT, VT, R, TERMS>), C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_paged_stream<NB, KT, VT, R, TERMS>, a, min_tiles);
}

template <typename F>
auto by_cache_types(int kt, int vt, F f) {
  using Q4 = std::integral_constant<int, kTypeQ4_0>;
  using Q8 = std::integral_constant<int, kTypeQ8_0>;
  if (kt == kTypeQ4_0) return vt == kTypeQ4_0 ? f(Q4(), Q4()) : f(Q4(), Q8());
  return vt == kTypeQ4_0 ? f(Q8(), Q4()) : f(Q8(), Q8());
}

// fp32 operands take two terms; more than 8 rows per pass only with one term
// and up to 128 channels (accumulators and query fragments fill the registers)
template <int NB>
constexpr bool two_groups(int elem, int rows8) {
  return NB <= 4 && elem != kElemF32 && rows8 > 1;
}

#define BQ_PAGED_STREAM_INSTANTIATE(NB)                                                                            \
  template <>                                                                                                      \
  StreamShape stream_shape<NB>(int kt, int vt, int elem, int rows8) {                                              \
    return by_cache_types(kt, vt, [&](auto k, auto v) {                                                            \
      using C1 = Cfg<NB, k.value, v.value, 1, 1>;                                                                  \
      using C2 = Cfg<NB, k.value, v.value, 2, 1>;                                                                  \
      using C1F = Cfg<NB, k.value, v.value, 1, 2>;                                                                 \
      if (elem == kElemF32) return StreamShape{C1F::ROWS, C1F::TOK, C1F::kCtas};                                   \
      if (two_groups<NB>(elem, rows8)) return StreamShape{C2::ROWS, C2::TOK, C2::kCtas};                           \
      return StreamShape{C1::ROWS, C1::TOK, C1::kCtas};                                                            \
    });                                                                                                            \
  }                                                                                                                \
  template <>                                                                                                      \
  cudaError_t launch_stream<NB>(const PagedAttnArgs &a, int rows8, int grid, int min_tiles, bool beside,           \
                                cudaStream_t stream) {                                                             \
    return by_cache_types(a.kt, a.vt, [&](auto k, auto v) {                                                        \
      if (a.elem == kElemF32)                                                                                      \
        return launch_stream_one<NB, k.value, v.value, 1, 2>(a, grid, min_tiles, beside, stream);                  \
      if constexpr (NB <= 4) {                                                                                     \
        if (rows8 > 1) return launch_stream_one<NB, k.value, v.value, 2, 1>(a, grid, min_tiles, beside, stream);   \
      }                                                                                                            \
      return launch_stream_one<NB, k.value, v.value, 1, 1>(a, grid, min_tiles, beside, stream);                    \
    });                                                                                                            \
  }

}  // namespace paged
}  // namespace bq

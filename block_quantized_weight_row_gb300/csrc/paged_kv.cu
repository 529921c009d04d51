// paged_kv.cu — the quantizing write into a paged KV cache, and reading token
// rows back.
//
// Write: K rows are optionally rotated (H64 / 8 per 64 channels, fp32
// butterflies of span 1, 2, ..., 32) and mean-centred (one fp32 subtraction),
// then each 32 channels become codes c = clamp(rne(x / d)) with d =
// binary16(amax / qmax), the rule of the contiguous cache write, bit for bit
// (lpnh.cn KV-cache article, §解法 and §三步上手; the pages describe one
// contiguous cache; slots into shared pages are this library's form). Read:
// d * c in fp32, plus the bias, out of the basis (H64 / 8 is its own inverse),
// rounded once to the output type.
//
// The floor is HBM: 2 or 4 bytes per value on one side and 0.56 or 1.06 on the
// other, against ~10 instructions per value to quantize. Write: 2 lanes per
// block (below), the next block's loads in flight. Read: 4 lanes per row, the
// next row's loads in flight. K and V are the two halves of one grid (a decode
// step's write is one launch); each half alone is as many CTAs as fit at once,
// so that V's start where K's leave.
// Measured, a layer of 32768 rows of 8 x 128 fp32 values, K in 4 (mean-centred)
// and V in 8 bits: write 58 us (5.6 TB/s of its 323 MB, 0.83 of the copy rate),
// read 61 us (5.3 TB/s): HBM and the latency of loads, 47 and 36 % of the SMs'
// warp slots in use. 65536 rows of 16-bit values in 4 bits, as many bytes but
// twice the values: write from bf16 104 us plain, 117 rotated and centred, read
// to bf16 67 and 84 us (4.1 TB/s). Instructions bind there: that read issues 2.9
// times the fp32 one's, its issue slots are 60 % used and its DRAM 43 %. Before,
// with a block per thread in a grid as large as the rows, the write took 95 us,
// and the read 65 and 94.
#include <algorithm>

#include "bq_internal.h"
#include "paged.cuh"

namespace bq {
namespace {

constexpr int kThreads = 256;
// CTAs per SM, for K and as many for V. Write: 4 fit with fp32 rows (64 registers), 5 with 16-bit ones (48); the layer and
// the 65536 rotated rows above took 61 / 118 us at 2, 69 / 124 at 3, 60 / 117 at 4, 63 / 117 at 5, 61 / 116 at 8. Read: also
// the launch bounds' minimum (80 registers at 3, fewer and spilled above); 60 / 99 us at 1, 63 / 90 at 2, 61 / 86 at 3, 69 / 92
// at 4, 78 / 122 at 5.
constexpr int kWriteCtas = 4;
constexpr int kReadCtas = 3;

// n / d for n < 2^29 by a multiplication: m = ceil(2^(32 + s) / d) with 2^s <=
// d < 2^(s + 1) errs by less than d <= 2^(s + 1) in 2^(32 + s), so n m errs by
// less than 2^(30 + s), the quotient by less than 1 / d: exact. Powers of two (where m
// would be 2^32) shift by s alone.
struct FastDiv {
  uint32_t m, s, pow2;
};
FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(2) << s) <= d) ++s;
  if ((d & (d - 1)) == 0) return FastDiv{0, s, 1};
  return FastDiv{uint32_t(((uint64_t(1) << (32 + s)) + d - 1) / d), s, 0};
}
__device__ __forceinline__ uint32_t operator/(uint32_t n, const FastDiv &d) {
  return (d.pow2 ? n : __umulhi(n, d.m)) >> d.s;
}

struct Shape {
  PagedShape sh;
  FastDiv by_nb, by_kv, by_per;  // blocks per row, kv heads, read items per row
};

struct WriteSide {
  const uint8_t *src;  // rows: token_stride and head_stride bytes apart, channels contiguous
  int64_t token_stride, head_stride;
  const float *bias;  // n_kv x D or null
  PagedPool pool;
};

struct ReadSide {
  uint8_t *dst;  // n_tokens x n_kv x D, contiguous
  const float *bias;
  PagedPool pool;
};

// 8 values of a row, as they are in memory
template <int ELEM>
struct Eight {
  uint4 v[Elem<ELEM>::kBytes / 2];
};
template <int ELEM>
__device__ __forceinline__ Eight<ELEM> load8(const uint8_t *p) {
  Eight<ELEM> e;
#pragma unroll
  for (int i = 0; i < Elem<ELEM>::kBytes / 2; ++i) e.v[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
  return e;
}
template <int ELEM>
__device__ __forceinline__ void floats8(const Eight<ELEM> &e, float *x) {
#pragma unroll
  for (int i = 0; i < Elem<ELEM>::kBytes / 2; ++i) {
    const uint32_t w[4] = {e.v[i].x, e.v[i].y, e.v[i].z, e.v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (ELEM == kElemF32) {
        x[4 * i + k] = __uint_as_float(w[k]);
      } else {
        const float2 f = unpack_pair<ELEM>(w[k]);
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    }
  }
}

// A block's 32 channels are held by 2 lanes, 16 each: lane j of the pair has
// channels 8j .. 8j+7 as x[0..7] and 16 + 8j .. as x[8..15]. So each 16-byte
// load of the pair is one 32-byte sector, and both nibbles of a Q4_0 byte are
// in one lane.

// H64 x / 8 of two blocks (lane bit 0: channel bit 3, lane bit 1: channel bit
// 5): the same sums in the same order as the contiguous write's rotation,
// spans 1, 2, ..., 32. Spans 2 and up run on fp32 pairs; a difference is the
// fused s * v + partner with s = -1, which rounds once like it.
__device__ __forceinline__ void hadamard64_4lanes_of16(float (&x)[16]) {
  const int lane = threadIdx.x & 31;
  uint64_t P[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[8 * h + 2 * i], b = x[8 * h + 2 * i + 1];
      P[h][i] = pack2(__float_as_uint(__fadd_rn(a, b)), __float_as_uint(__fsub_rn(a, b)));
    }
    hadamard_pairs<4>(P[h]);          // spans 2, 4
    hadamard_cross<4>(P[h], 1, lane);  // span 8
  }
  const uint64_t m1 = pack2(__float_as_uint(-1.0f), __float_as_uint(-1.0f));
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // span 16
    const uint64_t t = P[0][i];
    P[0][i] = fadd2(t, P[1][i]);
    P[1][i] = ffma2(m1, P[1][i], t);
  }
  const uint64_t e2 = pack2(__float_as_uint(0.125f), __float_as_uint(0.125f));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    hadamard_cross<4>(P[h], 2, lane);  // span 32
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      P[h][i] = fmul2(P[h][i], e2);
      x[8 * h + 2 * i] = __uint_as_float(uint32_t(P[h][i]));
      x[8 * h + 2 * i + 1] = __uint_as_float(uint32_t(P[h][i] >> 32));
    }
  }
}

// Code bytes (q + 8 for Q4_0, q mod 256 for Q8_0) of 16 values as four words.
// The common path runs on fp32 pairs, per value the operations of code_of: the
// product by the reciprocal, the rounding addition of a magic number (its low
// byte is the code byte), and the distance from the integer. A value near a
// tie or a subnormal scale (whose rounding can leave the range) sends the
// lane's values through the exact path; the bits are the same.
template <int TYPE>
__device__ __forceinline__ void codes_of16(const float (&x)[16], float ds, float inv, uint32_t (&w)[4]) {
  constexpr float kMagic = 12582912.0f + float(TYPE == kTypeQ4_0 ? 8 : 0);
  const uint64_t inv2 = pack2(__float_as_uint(inv), __float_as_uint(inv));
  const uint64_t mg2 = pack2(__float_as_uint(kMagic), __float_as_uint(kMagic));
  const uint64_t nmg2 = pack2(__float_as_uint(-kMagic), __float_as_uint(-kMagic));
  const uint64_t m1 = pack2(__float_as_uint(-1.0f), __float_as_uint(-1.0f));
  float far = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t t[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t r = fmul2(pack2(__float_as_uint(x[4 * q + 2 * k]), __float_as_uint(x[4 * q + 2 * k + 1])), inv2);
      const uint64_t tt = fadd2(r, mg2);
      const uint64_t e = ffma2(m1, fadd2(tt, nmg2), r);
      t[2 * k] = uint32_t(tt);
      t[2 * k + 1] = uint32_t(tt >> 32);
      far = fmaxf(far, fmaxf(fabsf(__uint_as_float(uint32_t(e))), fabsf(__uint_as_float(uint32_t(e >> 32)))));
    }
    w[q] = pack_bytes(t[0], t[1], t[2], t[3]);
  }
  if (far > 0.4999f || (ds > 0.0f && ds < 6.103515625e-05f)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t t[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] = uint32_t(code_of<TYPE>(x[4 * q + k], ds, inv) + (TYPE == kTypeQ4_0 ? 8 : 0));
      w[q] = pack_bytes(t[0], t[1], t[2], t[3]);
    }
  }
}

// A block on its way: this lane's 16 values, where they belong and the slot.
template <int ELEM>
struct Incoming {
  Eight<ELEM> lo, hi;
  uint32_t head, block;
  int64_t slot;
};
template <int ELEM>
__device__ __forceinline__ Incoming<ELEM> fetch_block(const WriteSide &s, const Shape &shape, const int64_t *slots, uint32_t i,
                                                      uint32_t n_blocks) {
  const uint32_t nb = uint32_t(shape.sh.nb), n_kv = uint32_t(shape.sh.n_kv), j = threadIdx.x & 1;
  const bool in = i < n_blocks;
  const uint32_t row = in ? i / shape.by_nb : 0, token = row / shape.by_kv;
  Incoming<ELEM> b;
  b.block = in ? i - row * nb : 0;
  b.head = row - token * n_kv;
  const uint8_t *src =
      s.src + int64_t(token) * s.token_stride + int64_t(b.head) * s.head_stride + (b.block * 32 + j * 8) * Elem<ELEM>::kBytes;
  b.lo = load8<ELEM>(src);
  b.hi = load8<ELEM>(src + 16 * Elem<ELEM>::kBytes);
  b.slot = __ldg(slots + token);
  if (!in) b.slot = -1;
  return b;
}

// Quantizes and stores it; every lane of the warp calls it.
template <int TYPE, int ELEM, bool ROT, bool IS_V>
__device__ __forceinline__ void write_block(const WriteSide &s, const Shape &shape, const Incoming<ELEM> &from, unsigned *err) {
  const PagedShape &sh = shape.sh;
  const uint32_t j = threadIdx.x & 1, nb = uint32_t(sh.nb), bl = from.block, head = from.head;
  const int64_t slot = from.slot;
  float x[16];
  floats8<ELEM>(from.lo, x);
  floats8<ELEM>(from.hi, x + 8);
  if constexpr (ROT) hadamard64_4lanes_of16(x);
  if (!IS_V && s.bias) {
    const float4 *b = reinterpret_cast<const float4 *>(s.bias + (head * nb + bl) * 32 + j * 8);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 p = __ldg(b + 4 * h), q = __ldg(b + 4 * h + 1);
      const float f[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) x[8 * h + k] = __fsub_rn(x[8 * h + k], f[k]);
    }
  }
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(x[k]));
  m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
  uint16_t scale;
  float ds;
  block_scale<TYPE>(m, scale, ds);
  uint32_t w[4];
  codes_of16<TYPE>(x, ds, ds > 0.0f ? rcp_approx(ds) : 0.0f, w);

  const SlotKind kind = slot_kind(sh, slot);
  if (kind == SlotKind::kBad && j == 0 && bl == 0) atomicOr(err, kErrIndex);
  const bool live = kind == SlotKind::kRow;
  uint32_t page, place;
  split_slot(sh, live ? uint32_t(slot) : 0u, page, place);
  uint8_t *hp = s.pool.base + (int64_t(page) * sh.n_kv + head) * s.pool.head_bytes;
  uint8_t *row = hp + int64_t(place) * s.pool.row_bytes;
  const bool odd = bl & 1, pair = (nb & 1) == 0;  // pair: blocks 2k, 2k+1 sit in lanes 2 apart
  if constexpr (TYPE == kTypeQ4_0) {
    const uint32_t w0 = w[0] | (w[2] << 4), w1 = w[1] | (w[3] << 4);  // code bytes 8j.., 8j + 4..
    if constexpr (!IS_V) {
      if (live) {
        uint32_t *o = reinterpret_cast<uint32_t *>(row);
        o[(2 * j) * nb + bl] = w0;
        o[(2 * j + 1) * nb + bl] = w1;
      }
    } else {
      // half-words 4j .. 4j+3; with the neighbouring block's lane, whole words:
      // the even block's lane takes the first two of both, the odd one's the others
      const uint32_t other = __shfl_xor_sync(kFull, odd ? w0 : w1, 2);
      if (live) {
        uint16_t *h = reinterpret_cast<uint16_t *>(row);
        if (pair) {
          const uint32_t a = odd ? other : w0, b = odd ? w1 : other, g = 4 * j + (odd ? 2 : 0), at = bl & ~1u;
          *reinterpret_cast<uint32_t *>(h + g * nb + at) = __byte_perm(a, b, 0x5410);
          *reinterpret_cast<uint32_t *>(h + (g + 1) * nb + at) = __byte_perm(a, b, 0x7632);
        } else {
          h[(4 * j) * nb + bl] = uint16_t(w0);
          h[(4 * j + 1) * nb + bl] = uint16_t(w0 >> 16);
          h[(4 * j + 2) * nb + bl] = uint16_t(w1);
          h[(4 * j + 3) * nb + bl] = uint16_t(w1 >> 16);
        }
      }
    }
  } else {
    if constexpr (!IS_V) {
      if (live) {
        uint2 *o = reinterpret_cast<uint2 *>(row);
        o[j * nb + bl] = make_uint2(w[0], w[1]);
        o[(2 + j) * nb + bl] = make_uint2(w[2], w[3]);
      }
    } else {
      // words of units 2j, 2j + 1, 4 + 2j, 5 + 2j, shared out likewise
      const uint32_t o0 = __shfl_xor_sync(kFull, odd ? w[0] : w[2], 2), o1 = __shfl_xor_sync(kFull, odd ? w[1] : w[3], 2);
      if (live) {
        uint32_t *h = reinterpret_cast<uint32_t *>(row);
        if (pair) {
          const uint32_t g = 2 * j + (odd ? 4 : 0), at = bl & ~1u;
          *reinterpret_cast<uint2 *>(h + g * nb + at) = odd ? make_uint2(o0, w[2]) : make_uint2(w[0], o0);
          *reinterpret_cast<uint2 *>(h + (g + 1) * nb + at) = odd ? make_uint2(o1, w[3]) : make_uint2(w[1], o1);
        } else {
          h[(2 * j) * nb + bl] = w[0];
          h[(2 * j + 1) * nb + bl] = w[1];
          h[(4 + 2 * j) * nb + bl] = w[2];
          h[(5 + 2 * j) * nb + bl] = w[3];
        }
      }
    }
  }
  if (live && j == 0) reinterpret_cast<uint16_t *>(hp + s.pool.scale_off)[place * nb + bl] = scale;
}

// Bound by HBM where there is enough of it: a thread fetches its next block
// before it quantizes this one (a block per thread and grid-sized launches left
// the memory waiting for CTAs to start: 95 us for the fp32 layer above; 8 values
// per lane paid the fixed costs twice: 65536 x 8 x 128 rotated bf16 144 us, 117
// so).
template <int KT, int VT, int ELEM, bool ROT>
__global__ void __launch_bounds__(kThreads)
    k_paged_write(const __grid_constant__ WriteSide k, const __grid_constant__ WriteSide v, const __grid_constant__ Shape sh,
                  const int64_t *__restrict__ slots, uint32_t n_blocks, unsigned *err) {
  // the 16 pairs of a warp are consecutive blocks and its trips uniform: every
  // lane stays, as pairs exchange values
  const uint32_t step = gridDim.x * (kThreads / 2);
  uint32_t i = (blockIdx.x * kThreads + threadIdx.x) / 2, warp0 = i & ~15u;
  if (warp0 >= n_blocks) return;
  const bool is_v = blockIdx.y != 0;
  Incoming<ELEM> now = fetch_block<ELEM>(is_v ? v : k, sh, slots, i, n_blocks);
  for (;;) {
    i += step;
    warp0 += step;
    const bool more = warp0 < n_blocks;
    const Incoming<ELEM> next = fetch_block<ELEM>(is_v ? v : k, sh, slots, i, more ? n_blocks : 0);
    if (is_v)
      write_block<VT, ELEM, false, true>(v, sh, now, err);
    else
      write_block<KT, ELEM, ROT, false>(k, sh, now, err);
    if (!more) break;
    now = next;
  }
}

// ------------------------------------------------------------------ read --

// One lane's 8 channels of a block, d * code in fp32: K lane c of 4 has unit c
// (Q4_0: channels 4c.., 16 + 4c..; Q8_0: channels 8c ..); a V lane takes units
// 2c and 2c + 1, which are the same channels. A code's bits under the exponent
// of 2^23 are 2^23 + u 16^k, exactly, for the nibble k of a half-word (or 2^23 +
// u for a byte); the subtraction leaves (u - 8) 16^k, and d 16^-k scales it, all
// without a rounding that d * (u - 8) would not have. Two instructions a value
// in place of shift, mask, subtract, convert, multiply.
template <int TYPE>
__device__ __forceinline__ void decode8(uint2 w, float d, float (&x)[8]) {
  auto pair = [&](uint32_t a, uint32_t b, float zero, float scale, float &lo, float &hi) {
    const uint64_t z2 = pack2(__float_as_uint(-zero), __float_as_uint(-zero)), s2 = pack2(__float_as_uint(scale), __float_as_uint(scale));
    const uint64_t v = fmul2(fadd2(pack2(a, b), z2), s2);
    lo = __uint_as_float(uint32_t(v));
    hi = __uint_as_float(uint32_t(v >> 32));
  };
  if constexpr (TYPE == kTypeQ4_0) {
    const uint32_t a = w.x, b = w.x >> 16;  // bytes 0, 1 and 2, 3: channels i and i + 2
    constexpr uint32_t E = 0x4b000000u;
    pair((a & 0xfu) | E, (b & 0xfu) | E, 8388608.0f + 8.0f, d, x[0], x[2]);
    pair((a & 0xf0u) | E, (b & 0xf0u) | E, 8388608.0f + 128.0f, d * 0.0625f, x[4], x[6]);
    pair((a & 0xf00u) | E, (b & 0xf00u) | E, 8388608.0f + 2048.0f, d * 0.00390625f, x[1], x[3]);
    pair((a & 0xf000u) | E, (b & 0xf000u) | E, 8388608.0f + 32768.0f, d * 0.000244140625f, x[5], x[7]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t u = (h ? w.y : w.x) ^ 0x80808080u;
      pair(__byte_perm(u, 0x4b000000u, 0x7440), __byte_perm(u, 0x4b000000u, 0x7441), 8388608.0f + 128.0f, d, x[4 * h], x[4 * h + 1]);
      pair(__byte_perm(u, 0x4b000000u, 0x7442), __byte_perm(u, 0x4b000000u, 0x7443), 8388608.0f + 128.0f, d, x[4 * h + 2], x[4 * h + 3]);
    }
  }
}

// The raw bytes of W blocks (b0 .. b0 + W - 1) of one token row, lane c's
// share: K its unit, V the units 2c and 2c + 1 (the same channels).
template <int TYPE, bool IS_V, int W>
struct Raw {
  static constexpr int UB = Codes<TYPE>::kBytes / (IS_V ? kUnitsV : kUnitsK);  // bytes of a unit: 4 or 8 (K), 2 or 4 (V)
  static constexpr int PIECE = UB * W, UNITS = IS_V ? 2 : 1;
  uint32_t code[UNITS][(PIECE + 3) / 4], scale[(W + 1) / 2];
};

template <int N>
__device__ __forceinline__ void load_raw(const uint8_t *p, uint32_t (&w)[(N + 3) / 4]) {
  if constexpr (N % 16 == 0) {
#pragma unroll
    for (int k = 0; k < N / 16; ++k) {
      const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(p) + k);
      w[4 * k] = q.x, w[4 * k + 1] = q.y, w[4 * k + 2] = q.z, w[4 * k + 3] = q.w;
    }
  } else if constexpr (N == 8) {
    const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(p));
    w[0] = q.x, w[1] = q.y;
  } else if constexpr (N == 4) {
    w[0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
  } else {
    static_assert(N == 2, "piece");
    w[0] = __ldcs(reinterpret_cast<const uint16_t *>(p));
  }
}

// Row and first block of a read item, the slot and whether it is a row.
struct ReadItem {
  uint32_t token, head, b0;
  bool in, live;
};
template <int W>
__device__ __forceinline__ ReadItem read_item(const Shape &shape, uint32_t item, uint32_t n_items) {
  const uint32_t nb = uint32_t(shape.sh.nb), n_kv = uint32_t(shape.sh.n_kv);
  ReadItem it;
  it.in = item < n_items;
  const uint32_t row = it.in ? item / shape.by_per : 0;
  it.b0 = it.in ? (item - row * (nb / W)) * W : 0;
  it.token = row / shape.by_kv;
  it.head = row - it.token * n_kv;
  it.live = false;
  return it;
}

// Where there is nothing to read (the last items, skipped and wrong slots) the
// pool's first row stands in. Wrong slots are reported.
template <int TYPE, bool IS_V, int W>
__device__ __forceinline__ Raw<TYPE, IS_V, W> read_raw(const ReadSide &s, const PagedShape &sh, ReadItem &it, int64_t slot, unsigned *err) {
  using R = Raw<TYPE, IS_V, W>;
  const uint32_t c = threadIdx.x & 3, nb = uint32_t(sh.nb);
  const SlotKind kind = it.in ? slot_kind(sh, slot) : SlotKind::kSkip;
  it.live = kind == SlotKind::kRow;
  if (kind == SlotKind::kBad) atomicOr(err, kErrIndex);
  uint32_t page, place;
  split_slot(sh, it.live ? uint32_t(slot) : 0u, page, place);
  const uint8_t *hp = s.pool.base + (int64_t(page) * sh.n_kv + it.head) * s.pool.head_bytes;
  const uint8_t *r = hp + int64_t(place) * s.pool.row_bytes;
  R raw;
#pragma unroll
  for (int h = 0; h < R::UNITS; ++h) load_raw<R::PIECE>(r + ((R::UNITS * c + h) * nb + it.b0) * R::UB, raw.code[h]);
  load_raw<2 * W>(hp + s.pool.scale_off + (place * nb + it.b0) * 2, raw.scale);
  return raw;
}

// Decodes an item and stores its rows; every lane of the warp calls it.
template <int TYPE, int ELEM, bool ROT, bool IS_V, int W>
__device__ __forceinline__ void read_store(const ReadSide &s, const Shape &shape, const ReadItem &it, const Raw<TYPE, IS_V, W> &raw) {
  using R = Raw<TYPE, IS_V, W>;
  const int c = threadIdx.x & 3;
  const uint32_t nb = uint32_t(shape.sh.nb), n_kv = uint32_t(shape.sh.n_kv);
  float x[W][8];
#pragma unroll
  for (int k = 0; k < W; ++k) {
    uint2 w;
    if constexpr (TYPE == kTypeQ4_0) {
      w.x = IS_V ? ((raw.code[0][k / 2] >> (16 * (k & 1))) & 0xffffu) | ((raw.code[R::UNITS - 1][k / 2] >> (16 * (k & 1))) << 16)
                 : raw.code[0][k];
      w.y = 0;
    } else {
      w = IS_V ? make_uint2(raw.code[0][k], raw.code[R::UNITS - 1][k])
               : make_uint2(raw.code[0][2 * k % ((R::PIECE + 3) / 4)], raw.code[0][(2 * k + 1) % ((R::PIECE + 3) / 4)]);
    }
    decode8<TYPE>(w, half_bits_to_float(raw.scale[k / 2] >> (16 * (k & 1))), x[k]);
  }
  if (!IS_V && s.bias) {
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 b =
            __ldg(reinterpret_cast<const float4 *>(s.bias + (it.head * nb + it.b0 + k) * 32 + chan8<TYPE>(c, h)));
        x[k][4 * h] = __fadd_rn(x[k][4 * h], b.x);
        x[k][4 * h + 1] = __fadd_rn(x[k][4 * h + 1], b.y);
        x[k][4 * h + 2] = __fadd_rn(x[k][4 * h + 2], b.z);
        x[k][4 * h + 3] = __fadd_rn(x[k][4 * h + 3], b.w);
      }
  }
  if constexpr (ROT && W >= 2) {
#pragma unroll
    for (int k = 0; k < W; k += 2) hadamard64_4lanes<TYPE>(reinterpret_cast<float(&)[2][8]>(x[k]));
  }
  uint8_t *out = s.dst + (int64_t(it.token) * n_kv + it.head) * nb * 32 * Elem<ELEM>::kBytes;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    if (!it.live) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = 0.0f;
    }
    const int b = int(it.b0 + k) * 32;
    if constexpr (ELEM == kElemF32) {
      if (it.in) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          __stcs(reinterpret_cast<float4 *>(out + (b + chan8<TYPE>(c, h)) * 4),
                 make_float4(x[k][4 * h], x[k][4 * h + 1], x[k][4 * h + 2], x[k][4 * h + 3]));
      }
    } else {
      uint2 lo = make_uint2(pack_pair<ELEM>(x[k][0], x[k][1]), pack_pair<ELEM>(x[k][2], x[k][3]));
      uint2 hi = make_uint2(pack_pair<ELEM>(x[k][4], x[k][5]), pack_pair<ELEM>(x[k][6], x[k][7]));
      int at = b + 8 * c;
      if constexpr (TYPE == kTypeQ4_0) {
        // lanes 2k and 2k + 1 have 4 neighbouring channels of both halves of
        // the block: the even one takes the low half's 8, the odd the high's
        const bool odd = c & 1;
        const uint32_t ox = __shfl_xor_sync(kFull, odd ? lo.x : hi.x, 1), oy = __shfl_xor_sync(kFull, odd ? lo.y : hi.y, 1);
        const uint2 other = make_uint2(ox, oy);
        if (odd)
          lo = other;
        else
          hi = other;
        at = b + (odd ? 16 : 0) + 8 * (c >> 1);
      }
      if (it.in) __stcs(reinterpret_cast<uint4 *>(out + at * 2), make_uint4(lo.x, lo.y, hi.x, hi.y));
    }
  }
}

// A lane's items, `step` apart: the next one's bytes and the slot of the one
// after that are on their way while this one is decoded and stored.
template <int TYPE, int ELEM, bool ROT, bool IS_V, int W>
__device__ __forceinline__ void read_side(const ReadSide &s, const Shape &shape, const int64_t *slots, uint32_t item, uint32_t step,
                                          uint32_t n_items, unsigned *err) {
  uint32_t warp0 = item & ~7u;  // a warp's 8 groups of 4 lanes are consecutive items, its trips uniform
  if (warp0 >= n_items) return;
  ReadItem it = read_item<W>(shape, item, n_items), it1 = read_item<W>(shape, item + step, n_items);
  int64_t slot1 = __ldg(slots + it1.token);
  Raw<TYPE, IS_V, W> raw = read_raw<TYPE, IS_V, W>(s, shape.sh, it, __ldg(slots + it.token), err);
  for (;;) {
    const Raw<TYPE, IS_V, W> raw1 = read_raw<TYPE, IS_V, W>(s, shape.sh, it1, slot1, err);
    const ReadItem it2 = read_item<W>(shape, item + 2 * step, n_items);
    const int64_t slot2 = __ldg(slots + it2.token);
    read_store<TYPE, ELEM, ROT, IS_V, W>(s, shape, it, raw);
    item += step;
    warp0 += step;
    if (warp0 >= n_items) return;
    it = it1;
    raw = raw1;
    it1 = it2;
    slot1 = slot2;
  }
}

template <int KT, int VT, int ELEM, bool ROT, int W>
__global__ void __launch_bounds__(kThreads, kReadCtas)
    k_paged_read(const __grid_constant__ ReadSide k, const __grid_constant__ ReadSide v, const __grid_constant__ Shape sh,
                 const int64_t *__restrict__ slots, uint32_t n_items, unsigned *err) {
  const uint32_t item = (blockIdx.x * kThreads + threadIdx.x) / 4, step = gridDim.x * (kThreads / 4);
  if (blockIdx.y == 0)
    read_side<KT, ELEM, ROT, false, W>(k, sh, slots, item, step, n_items, err);
  else
    read_side<VT, ELEM, false, true, W>(v, sh, slots, item, step, n_items, err);
}

// calls f with compile-time K type, V type and element type
template <typename F>
cudaError_t by_types(int kt, int vt, int elem, F f) {
  auto on_elem = [&](auto k, auto v) {
    switch (elem) {
      case kElemF32: return f(k, v, std::integral_constant<int, kElemF32>());
      case kElemF16: return f(k, v, std::integral_constant<int, kElemF16>());
      default: return f(k, v, std::integral_constant<int, kElemBF16>());
    }
  };
  using Q4 = std::integral_constant<int, kTypeQ4_0>;
  using Q8 = std::integral_constant<int, kTypeQ8_0>;
  if (kt == kTypeQ4_0) return vt == kTypeQ4_0 ? on_elem(Q4(), Q4()) : on_elem(Q4(), Q8());
  return vt == kTypeQ4_0 ? on_elem(Q8(), Q4()) : on_elem(Q8(), Q8());
}

// tokens per launch, so that block indexes stay within 32 bits
int64_t token_chunk(const PagedShape &sh) { return std::max<int64_t>(1, (int64_t(1) << 29) / (int64_t(sh.n_kv) * sh.nb)); }

}  // namespace

cudaError_t launch_paged_write(const PagedPool &kp, const PagedPool &vp, const PagedShape &sh, int kt, int vt, int elem,
                               bool rotate, const void *K, int64_t k_ts, int64_t k_hs, const void *V, int64_t v_ts,
                               int64_t v_hs, const float *bias, const int64_t *slots, int64_t n_tokens,
                               cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  const Shape shape{sh, fast_div(uint32_t(sh.nb)), fast_div(uint32_t(sh.n_kv)), fast_div(1)};
  const int64_t chunk = token_chunk(sh);
  for (int64_t t = 0; t < n_tokens; t += chunk) {
    const uint32_t n_blocks = uint32_t(std::min(chunk, n_tokens - t) * sh.n_kv * sh.nb);
    const WriteSide k{static_cast<const uint8_t *>(K) + t * k_ts, k_ts, k_hs, bias, kp};
    const WriteSide v{static_cast<const uint8_t *>(V) + t * v_ts, v_ts, v_hs, nullptr, vp};
    // a half as large as what is resident, with several blocks per thread
    const uint32_t ctas = (n_blocks + kThreads / 2 - 1) / (kThreads / 2);
    const dim3 grid(std::min<uint32_t>(ctas, uint32_t(di->sm_count) * kWriteCtas), 2);
    err = by_types(kt, vt, elem, [&](auto k_, auto v_, auto e_) {
      if (rotate)
        k_paged_write<k_.value, v_.value, e_.value, true><<<grid, kThreads, 0, stream>>>(k, v, shape, slots + t, n_blocks, di->err_word);
      else
        k_paged_write<k_.value, v_.value, e_.value, false><<<grid, kThreads, 0, stream>>>(k, v, shape, slots + t, n_blocks, di->err_word);
      return cudaGetLastError();
    });
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t launch_paged_read(const PagedPool &kp, const PagedPool &vp, const PagedShape &sh, int kt, int vt, int elem,
                              bool rotate, void *K, void *V, const float *bias, const int64_t *slots, int64_t n_tokens,
                              cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  const int64_t chunk = token_chunk(sh), es = elem == kElemF32 ? 4 : 2;
  const int W = sh.nb % 4 == 0 ? 4 : sh.nb % 2 == 0 ? 2 : 1;
  const Shape shape{sh, fast_div(uint32_t(sh.nb)), fast_div(uint32_t(sh.n_kv)), fast_div(uint32_t(sh.nb / W))};
  if (sh.n_pages == 0) return cudaErrorInvalidValue;  // refused by the ABI layer: no row to stand in
  for (int64_t t = 0; t < n_tokens; t += chunk) {
    const uint32_t n_items = uint32_t(std::min(chunk, n_tokens - t) * sh.n_kv * (sh.nb / W));
    const int64_t off = t * sh.n_kv * sh.nb * 32 * es;
    const ReadSide k{static_cast<uint8_t *>(K) + off, bias, kp}, v{static_cast<uint8_t *>(V) + off, nullptr, vp};
    const uint32_t ctas = (n_items + kThreads / 4 - 1) / (kThreads / 4);
    const dim3 grid(std::min<uint32_t>(ctas, uint32_t(di->sm_count) * kReadCtas), 2);
    err = by_types(kt, vt, elem, [&](auto k_, auto v_, auto e_) {
      auto go = [&](auto rot, auto w) {
        k_paged_read<k_.value, v_.value, e_.value, rot.value, w.value><<<grid, kThreads, 0, stream>>>(k, v, shape, slots + t, n_items, di->err_word);
        return cudaGetLastError();
      };
      using W1 = std::integral_constant<int, 1>;
      using W2 = std::integral_constant<int, 2>;
      using W4 = std::integral_constant<int, 4>;
      if (rotate) return W == 4 ? go(std::true_type(), W4()) : go(std::true_type(), W2());
      return W == 4 ? go(std::false_type(), W4()) : W == 2 ? go(std::false_type(), W2()) : go(std::false_type(), W1());
    });
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace bq

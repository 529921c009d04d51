// paged.cuh — the page layout of the paged KV cache and the element types its
// operators read and write.
//
// A pool is n_pages x n_kv_heads "head pages" of page_size tokens. The bytes
// of a head page are two planes: the codes of its tokens, row after row, then
// their binary16 scales [place][block]. A block of 32 channels has the code
// bytes of the Q4_0 or Q8_0 block (the pages name both as cache types: "05.
// llama.cpp：从 GGUF 文件到本地推理服务", §KV Cache 类型与 Flash Attention), so
// that a head page holds exactly the bytes per value of the blocks; only their
// order differs. The code bytes of a block are cut into 4 units (K) or 8 units
// (V), and a row is unit 0 of every block, unit 1 of every block, and so on:
// with m16n8k16 fragments (attention), lane quad c contracts over unit c of a
// K row, and lane group g owns the channels of unit g of a V row, so each lane
// reads its share of a row as one piece, 16-byte aligned rows, no block
// straddling a word (an 18-byte block starts on an odd half-word every time).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bq_device.cuh"

namespace bq {

constexpr int kPagedTile = 16;  // tokens of one matrix-instruction tile; page sizes are multiples of it
constexpr int kUnitsK = 4, kUnitsV = 8;

template <int TYPE> struct Codes;
template <> struct Codes<kTypeQ4_0> { static constexpr int kBytes = 16; };
template <> struct Codes<kTypeQ8_0> { static constexpr int kBytes = 32; };

// One tensor's pool. Token rows are addressed by slot = page * page_size + place.
struct PagedPool {
  uint8_t *base;
  int64_t head_bytes;   // bytes of one head page
  int64_t scale_off;    // byte offset of its scales
  int row_bytes;        // bytes of one token's codes
};

struct PagedShape {
  int64_t n_pages;
  int page_size, page_shift;  // shift: log2(page_size), or -1
  uint64_t page_magic;        // ceil(2^64 / (page_size / 16)), for page sizes that are no power of two
  int n_kv, nb;               // kv heads, blocks of 32 channels per head
};

__host__ __device__ __forceinline__ void split_slot(const PagedShape &s, uint32_t slot, uint32_t &page, uint32_t &place) {
  page = s.page_shift >= 0 ? slot >> s.page_shift : slot / uint32_t(s.page_size);
  place = slot - page * uint32_t(s.page_size);
}

// Page number of a sequence's token, without a branch (one would make loads
// in flight wait where it ends). token < 2^31: token / 16 < 2^27 and
// page_size / 16 <= 2^16, so the product with the rounded-up reciprocal errs
// by less than 2^43 / 2^64 and the quotient is exact.
__device__ __forceinline__ int token_page(const PagedShape &s, int token) {
  const int by_shift = token >> (s.page_shift & 31), by_magic = int(__umul64hi(uint64_t(token >> 4), s.page_magic));
  return s.page_shift >= 0 ? by_shift : by_magic;
}

// A slot of the caller: a row of the pool, skipped (-1), or neither. Slots
// are checked here, in 64 bits, before any address is made of them.
enum class SlotKind { kRow, kSkip, kBad };
__host__ __device__ __forceinline__ SlotKind slot_kind(const PagedShape &s, int64_t slot) {
  if (slot == -1) return SlotKind::kSkip;
  return slot >= 0 && slot < s.n_pages * s.page_size ? SlotKind::kRow : SlotKind::kBad;
}

// ------------------------------------------------------- element types --

constexpr int kElemF32 = 0, kElemF16 = 1, kElemBF16 = 2;

template <int ELEM> struct Elem;
template <> struct Elem<kElemF32> { static constexpr int kBytes = 4; };
template <> struct Elem<kElemF16> { static constexpr int kBytes = 2; };
template <> struct Elem<kElemBF16> { static constexpr int kBytes = 2; };

// two 16-bit values of a word as fp32
template <int ELEM>
__device__ __forceinline__ float2 unpack_pair(uint32_t w) {
  if constexpr (ELEM == kElemF16) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
}

template <int ELEM>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  if constexpr (ELEM == kElemF16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

// 4 lanes share a block of 32 channels: lane c has the 8 channels of K unit c.
// First channel of its values 0-3 (half 0) and 4-7 (half 1).
template <int TYPE>
__device__ __forceinline__ int chan8(int c, int half) {
  return TYPE == kTypeQ4_0 ? 4 * c + 16 * half : 8 * c + 4 * half;
}

// Butterflies on fp32 pairs. In the lane: (P[i], P[i + h]) -> sum, difference
// for h = 1, 2, .. N / 2 pairs; across lanes: lanes m apart.
template <int N>
__device__ __forceinline__ void hadamard_pairs(uint64_t (&P)[N]) {
  const uint64_t m1 = pack2(__float_as_uint(-1.0f), __float_as_uint(-1.0f));
#pragma unroll
  for (int h = 1; h < N; h <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & h) == 0) {
        const uint64_t t = P[i];
        P[i] = fadd2(t, P[i + h]);
        P[i + h] = ffma2(m1, P[i + h], t);
      }
}
template <int N>
__device__ __forceinline__ void hadamard_cross(uint64_t (&P)[N], int m, int lane) {
  const float s = (lane & m) ? -1.0f : 1.0f;
  const uint64_t s2 = pack2(__float_as_uint(s), __float_as_uint(s));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t lo = __shfl_xor_sync(kFull, uint32_t(P[i]), m), hi = __shfl_xor_sync(kFull, uint32_t(P[i] >> 32), m);
    P[i] = ffma2(s2, P[i], pack2(lo, hi));
  }
}

// The butterflies of a 64-channel group held by 4 lanes (two blocks x 8
// values each), spans in order 1, 2, ..., 32, then 1/8.
template <int TYPE>
__device__ __forceinline__ void hadamard64_4lanes(float (&x)[2][8]) {
  const int lane = threadIdx.x & 31;
  uint64_t P[2][4];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
#pragma unroll
    for (int i = 0; i < 4; ++i)  // span 1
      P[b][i] = pack2(__float_as_uint(__fadd_rn(x[b][2 * i], x[b][2 * i + 1])), __float_as_uint(__fsub_rn(x[b][2 * i], x[b][2 * i + 1])));
    const uint64_t m1 = pack2(__float_as_uint(-1.0f), __float_as_uint(-1.0f));
    auto inner = [&](int h) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((i & h) == 0) {
          const uint64_t t = P[b][i];
          P[b][i] = fadd2(t, P[b][i + h]);
          P[b][i + h] = ffma2(m1, P[b][i + h], t);
        }
    };
    inner(1);  // span 2
    if constexpr (TYPE == kTypeQ4_0) {  // channel bits 2, 3 are the lane's, bit 4 the value's
      hadamard_cross<4>(P[b], 1, lane);
      hadamard_cross<4>(P[b], 2, lane);
      inner(2);
    } else {  // channel bit 2 is the value's, bits 3, 4 the lane's
      inner(2);
      hadamard_cross<4>(P[b], 1, lane);
      hadamard_cross<4>(P[b], 2, lane);
    }
  }
  const uint64_t e2 = pack2(__float_as_uint(0.125f), __float_as_uint(0.125f)), m1 = pack2(__float_as_uint(-1.0f), __float_as_uint(-1.0f));
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // span 32
    const uint64_t p = fmul2(fadd2(P[0][i], P[1][i]), e2), q = fmul2(ffma2(m1, P[1][i], P[0][i]), e2);
    x[0][2 * i] = __uint_as_float(uint32_t(p)), x[0][2 * i + 1] = __uint_as_float(uint32_t(p >> 32));
    x[1][2 * i] = __uint_as_float(uint32_t(q)), x[1][2 * i + 1] = __uint_as_float(uint32_t(q >> 32));
  }
}

}  // namespace bq

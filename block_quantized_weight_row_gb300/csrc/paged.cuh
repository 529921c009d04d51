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

// The butterflies of a 64-channel group held by 4 lanes (two blocks x 8
// values each), spans in order 1, 2, ..., 32, then 1/8.
template <int TYPE>
__device__ __forceinline__ void hadamard64_4lanes(float (&x)[2][8]) {
  const int lane = threadIdx.x & 31;
  auto inner = [&](int bit) {  // span within the lane: bit of the value index
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i & bit) == 0) {
          const float p = x[b][i], q = x[b][i + bit];
          x[b][i] = __fadd_rn(p, q);
          x[b][i + bit] = __fsub_rn(p, q);
        }
  };
  auto cross = [&](int m) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_xor_sync(kFull, x[b][i], m);
        x[b][i] = (lane & m) ? __fsub_rn(o, x[b][i]) : __fadd_rn(x[b][i], o);
      }
  };
  inner(1);
  inner(2);
  if constexpr (TYPE == kTypeQ4_0) {  // channel bits 2, 3 are the lane's, bit 4 the value's
    cross(1);
    cross(2);
    inner(4);
  } else {  // channel bit 2 is the value's, bits 3, 4 the lane's
    inner(4);
    cross(1);
    cross(2);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = x[0][i], q = x[1][i];
    x[0][i] = __fmul_rn(__fadd_rn(p, q), 0.125f);
    x[1][i] = __fmul_rn(__fsub_rn(p, q), 0.125f);
  }
}

}  // namespace bq

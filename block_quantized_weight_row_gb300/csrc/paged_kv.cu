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
// Both are bound by HBM: 2 or 4 bytes per value on one side and 0.56 or 1.06
// on the other, against ~15 instructions per value to quantize. Write: 4 lanes
// per block with 8 values each, so that 16-byte loads of a warp are one
// contiguous run without staging through shared memory; the amax takes two
// shuffles, the low and high nibbles meet by one more, spans 8-32 of the
// rotation one each. K and V are the two halves of one grid (a decode step's
// write is one launch).
#include <algorithm>

#include "bq_internal.h"
#include "paged.cuh"

namespace bq {
namespace {

constexpr int kThreads = 256;

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

template <int ELEM>
__device__ __forceinline__ void load8(const uint8_t *p, float (&v)[8]) {
  if constexpr (ELEM == kElemF32) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_pair<ELEM>(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// H64 x / 8 of 64 channels held 8 per lane by 8 consecutive lanes (lane j of
// the 8 holds channels 8j .. 8j+7): the same sums in the same order as the
// contiguous write's rotation.
__device__ __forceinline__ void hadamard64_8lanes_of8(float (&v)[8]) {
#pragma unroll
  for (int span = 1; span < 8; span <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & span) == 0) {
        const float a = v[i], b = v[i + span];
        v[i] = __fadd_rn(a, b);
        v[i + span] = __fsub_rn(a, b);
      }
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 1; m < 8; m <<= 1)  // spans 8, 16, 32
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_xor_sync(kFull, v[i], m);
      v[i] = (lane & m) ? __fsub_rn(o, v[i]) : __fadd_rn(v[i], o);
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], 0.125f);
}

// U blocks of this lane's groups of 4, `step` blocks apart; every lane of the
// warp calls it. All are loaded before the first is quantized.
template <int TYPE, int ELEM, bool ROT, bool IS_V, int U>
__device__ __forceinline__ void write_blocks(const WriteSide &s, const PagedShape &sh, const int64_t *slots,
                                             uint32_t first, uint32_t step, uint32_t n_blocks, unsigned *err) {
  const int j = threadIdx.x & 3;
  const uint32_t nb = uint32_t(sh.nb), n_kv = uint32_t(sh.n_kv);
  float v[U][8];
  int64_t slot[U];
  uint32_t head[U], block[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = first + u * step;
    slot[u] = -1;
    head[u] = block[u] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[u][k] = 0.0f;
    if (i < n_blocks) {
      const uint32_t row = i / nb, token = row / n_kv;
      block[u] = i - row * nb;
      head[u] = row - token * n_kv;
      slot[u] = __ldg(slots + token);
      load8<ELEM>(s.src + int64_t(token) * s.token_stride + int64_t(head[u]) * s.head_stride +
                      (block[u] * 32 + j * 8) * Elem<ELEM>::kBytes,
                  v[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float(&x)[8] = v[u];
    if constexpr (ROT) hadamard64_8lanes_of8(x);
    if (!IS_V && s.bias) {
      const float4 *b = reinterpret_cast<const float4 *>(s.bias + (head[u] * nb + block[u]) * 32 + j * 8);
      const float4 p = __ldg(b), q = __ldg(b + 1);
      const float f[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __fsub_rn(x[k], f[k]);
    }
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[k]));
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
    uint16_t scale;
    float ds;
    block_scale<TYPE>(m, scale, ds);
    const float inv = ds > 0.0f ? rcp_approx(ds) : 0.0f;
    uint32_t q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = uint32_t(code_of<TYPE>(x[k], ds, inv) + (TYPE == kTypeQ4_0 ? 8 : 0));
    const uint32_t a = pack_bytes(q[0], q[1], q[2], q[3]), b = pack_bytes(q[4], q[5], q[6], q[7]);

    const SlotKind kind = slot_kind(sh, slot[u]);
    if (kind == SlotKind::kBad && j == 0 && block[u] == 0) atomicOr(err, kErrIndex);
    const bool live = kind == SlotKind::kRow;
    uint32_t page = 0, place = 0;
    if (live) split_slot(sh, uint32_t(slot[u]), page, place);
    uint8_t *hp = s.pool.base + (int64_t(page) * sh.n_kv + head[u]) * s.pool.head_bytes;
    uint8_t *row = hp + int64_t(place) * s.pool.row_bytes;
    const uint32_t bl = block[u];
    const bool odd = bl & 1, pair = (nb & 1) == 0;  // pair: blocks 2k, 2k+1 sit in lanes 4 apart
    if constexpr (TYPE == kTypeQ4_0) {
      // code bytes 4c .. 4c+3: low nibbles of lane c / 2, high nibbles of lane c / 2 + 2
      const uint32_t got = __shfl_xor_sync(kFull, j < 2 ? b : a, 2);
      const uint32_t c = j < 2 ? 2 * j : 2 * (j - 2) + 1;
      const uint32_t w = j < 2 ? (a | (got << 4)) : (got | (b << 4));
      if constexpr (!IS_V) {
        if (live) reinterpret_cast<uint32_t *>(row)[c * nb + bl] = w;
      } else {
        // V: half-words 2c and 2c+1; with the neighbouring block's lane, one whole word each
        const uint32_t other = __shfl_xor_sync(kFull, odd ? w & 0xffffu : w >> 16, 4);
        if (live) {
          uint16_t *h = reinterpret_cast<uint16_t *>(row);
          if (pair) {
            const uint32_t g = 2 * c + odd;
            *reinterpret_cast<uint32_t *>(h + g * nb + (bl & ~1u)) =
                odd ? (other | (w & 0xffff0000u)) : ((w & 0xffffu) | (other << 16));
          } else {
            h[(2 * c) * nb + bl] = uint16_t(w);
            h[(2 * c + 1) * nb + bl] = uint16_t(w >> 16);
          }
        }
      }
    } else {
      if constexpr (!IS_V) {
        if (live) reinterpret_cast<uint2 *>(row)[j * nb + bl] = make_uint2(a, b);
      } else {
        const uint32_t other = __shfl_xor_sync(kFull, odd ? a : b, 4);
        if (live) {
          uint32_t *h = reinterpret_cast<uint32_t *>(row);
          if (pair) {
            const uint32_t g = 2 * j + odd;
            *reinterpret_cast<uint2 *>(h + g * nb + (bl & ~1u)) = odd ? make_uint2(other, b) : make_uint2(a, other);
          } else {
            h[(2 * j) * nb + bl] = a;
            h[(2 * j + 1) * nb + bl] = b;
          }
        }
      }
    }
    if (live && j == 0) reinterpret_cast<uint16_t *>(hp + s.pool.scale_off)[place * nb + bl] = scale;
  }
}

template <int KT, int VT, int ELEM, bool ROT>
__global__ void __launch_bounds__(kThreads)
    k_paged_write(const WriteSide k, const WriteSide v, const PagedShape sh, const int64_t *__restrict__ slots,
                  uint32_t n_blocks, unsigned *err) {
  constexpr int U = 2;
  const uint32_t step = gridDim.x * (kThreads / 4);
  // the 8 groups of a warp are consecutive blocks, and a warp's trips are
  // uniform, so that every shuffle has all lanes
  const uint32_t group = (blockIdx.x * kThreads + threadIdx.x) / 4, warp0 = group & ~7u;
  for (uint32_t i = 0; warp0 + i < n_blocks; i += U * step) {
    if (blockIdx.y == 0)
      write_blocks<KT, ELEM, ROT, false, U>(k, sh, slots, group + i, step, n_blocks, err);
    else
      write_blocks<VT, ELEM, false, true, U>(v, sh, slots, group + i, step, n_blocks, err);
  }
}

// ------------------------------------------------------------------ read --

// 4 values at channel `at` of an output row
template <int ELEM>
__device__ __forceinline__ void store4(uint8_t *row, int at, const float (&x)[4]) {
  uint8_t *p = row + at * Elem<ELEM>::kBytes;
  if constexpr (ELEM == kElemF32)
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
  else
    __stcs(reinterpret_cast<uint2 *>(p), make_uint2(pack_pair<ELEM>(x[0], x[1]), pack_pair<ELEM>(x[2], x[3])));
}

// One lane's 8 channels of a block as fp32 codes: K lane c of 4 has unit c
// (Q4_0: channels 4c.., 16 + 4c..; Q8_0: channels 8c ..); a V lane takes units
// 2c and 2c + 1, which are the same channels.
template <int TYPE>
__device__ __forceinline__ void decode8(uint2 w, float d, float (&x)[8]) {
  if constexpr (TYPE == kTypeQ4_0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __fmul_rn(d, float(int((w.x >> (8 * i)) & 15u) - 8));
      x[4 + i] = __fmul_rn(d, float(int((w.x >> (8 * i + 4)) & 15u) - 8));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __fmul_rn(d, float(int8_t(w.x >> (8 * i))));
      x[4 + i] = __fmul_rn(d, float(int8_t(w.y >> (8 * i))));
    }
  }
}

// W blocks (b0 .. b0 + W - 1) of one token row by 4 lanes.
template <int TYPE, int ELEM, bool ROT, bool IS_V, int W>
__device__ __forceinline__ void read_blocks(const ReadSide &s, const PagedShape &sh, const int64_t *slots,
                                            uint32_t item, uint32_t n_items, unsigned *err) {
  const int c = threadIdx.x & 3;
  const uint32_t nb = uint32_t(sh.nb), n_kv = uint32_t(sh.n_kv), per = nb / W;
  const bool in = item < n_items;
  const uint32_t row = in ? item / per : 0, b0 = in ? (item - row * per) * W : 0;
  const uint32_t token = row / n_kv, head = row - token * n_kv;
  const int64_t slot = in ? __ldg(slots + token) : -1;
  const SlotKind kind = slot_kind(sh, slot);
  if (kind == SlotKind::kBad && c == 0 && b0 == 0) atomicOr(err, kErrIndex);
  uint2 w[W];
  float d[W];
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = make_uint2(TYPE == kTypeQ4_0 ? 0x88888888u : 0u, 0u), d[k] = 0.0f;
  if (kind == SlotKind::kRow) {
    uint32_t page, place;
    split_slot(sh, uint32_t(slot), page, place);
    const uint8_t *hp = s.pool.base + (int64_t(page) * sh.n_kv + head) * s.pool.head_bytes;
    const uint8_t *r = hp + int64_t(place) * s.pool.row_bytes;
    const uint16_t *sc = reinterpret_cast<const uint16_t *>(hp + s.pool.scale_off) + place * nb + b0;
    constexpr int UB = Codes<TYPE>::kBytes / (IS_V ? kUnitsV : kUnitsK);  // bytes of a unit: 4 or 8 (K), 2 or 4 (V)
    constexpr int PIECE = UB * W;                                         // bytes of a unit of W blocks
    // K: one piece; V: the pieces of units 2c and 2c + 1
    uint32_t raw[IS_V ? 2 : 1][(PIECE + 3) / 4];
#pragma unroll
    for (int h = 0; h < (IS_V ? 2 : 1); ++h) {
      const uint8_t *p = r + ((IS_V ? 2 * c + h : c) * nb + b0) * UB;
      if constexpr (PIECE >= 16) {
#pragma unroll
        for (int k = 0; k < PIECE / 16; ++k) {
          const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(p) + k);
          raw[h][4 * k] = q.x, raw[h][4 * k + 1] = q.y, raw[h][4 * k + 2] = q.z, raw[h][4 * k + 3] = q.w;
        }
      } else if constexpr (PIECE == 8) {
        const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(p));
        raw[h][0] = q.x, raw[h][1] = q.y;
      } else if constexpr (PIECE == 4) {
        raw[h][0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
      } else {
        raw[h][0] = __ldcs(reinterpret_cast<const uint16_t *>(p));
      }
    }
    if constexpr (W == 4) {
      const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(sc));
      d[0] = half_bits_to_float(q.x), d[1] = half_bits_to_float(q.x >> 16);
      d[2] = half_bits_to_float(q.y), d[3] = half_bits_to_float(q.y >> 16);
    } else if constexpr (W == 2) {
      const uint32_t q = __ldcs(reinterpret_cast<const uint32_t *>(sc));
      d[0] = half_bits_to_float(q), d[1] = half_bits_to_float(q >> 16);
    } else {
      d[0] = half_bits_to_float(__ldcs(sc));
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if constexpr (TYPE == kTypeQ4_0 && !IS_V)
        w[k].x = raw[0][k];
      else if constexpr (TYPE == kTypeQ4_0)
        w[k].x = ((raw[0][k / 2] >> (16 * (k & 1))) & 0xffffu) | ((raw[IS_V][k / 2] >> (16 * (k & 1))) << 16);
      else if constexpr (!IS_V)
        w[k] = make_uint2(raw[0][2 * k], raw[0][2 * k + 1]);
      else
        w[k] = make_uint2(raw[0][k], raw[IS_V][k]);
    }
  }
  float x[W][8];
#pragma unroll
  for (int k = 0; k < W; ++k) decode8<TYPE>(w[k], d[k], x[k]);
  if (!IS_V && s.bias && kind == SlotKind::kRow) {
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 b = __ldg(reinterpret_cast<const float4 *>(s.bias + (head * nb + b0 + k) * 32 + chan8<TYPE>(c, h)));
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
  if (!in) return;
  uint8_t *out = s.dst + (int64_t(token) * n_kv + head) * nb * 32 * Elem<ELEM>::kBytes;
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float y[4] = {x[k][4 * h], x[k][4 * h + 1], x[k][4 * h + 2], x[k][4 * h + 3]};
      store4<ELEM>(out, int(b0 + k) * 32 + chan8<TYPE>(c, h), y);
    }
}

template <int KT, int VT, int ELEM, bool ROT, int W>
__global__ void __launch_bounds__(kThreads)
    k_paged_read(const ReadSide k, const ReadSide v, const PagedShape sh, const int64_t *__restrict__ slots,
                 uint32_t n_items, unsigned *err) {
  const uint32_t item = (blockIdx.x * kThreads + threadIdx.x) / 4;
  if (blockIdx.y == 0)
    read_blocks<KT, ELEM, ROT, false, W>(k, sh, slots, item, n_items, err);
  else
    read_blocks<VT, ELEM, false, true, W>(v, sh, slots, item, n_items, err);
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
  const int64_t chunk = token_chunk(sh);
  for (int64_t t = 0; t < n_tokens; t += chunk) {
    const uint32_t n_blocks = uint32_t(std::min(chunk, n_tokens - t) * sh.n_kv * sh.nb);
    const WriteSide k{static_cast<const uint8_t *>(K) + t * k_ts, k_ts, k_hs, bias, kp};
    const WriteSide v{static_cast<const uint8_t *>(V) + t * v_ts, v_ts, v_hs, nullptr, vp};
    const uint32_t ctas = (n_blocks + kThreads / 4 - 1) / (kThreads / 4);
    const dim3 grid(std::min<uint32_t>(ctas, uint32_t(di->sm_count) * 32), 2);
    err = by_types(kt, vt, elem, [&](auto k_, auto v_, auto e_) {
      if (rotate)
        k_paged_write<k_.value, v_.value, e_.value, true><<<grid, kThreads, 0, stream>>>(k, v, sh, slots + t, n_blocks, di->err_word);
      else
        k_paged_write<k_.value, v_.value, e_.value, false><<<grid, kThreads, 0, stream>>>(k, v, sh, slots + t, n_blocks, di->err_word);
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
  for (int64_t t = 0; t < n_tokens; t += chunk) {
    const uint32_t n_items = uint32_t(std::min(chunk, n_tokens - t) * sh.n_kv * (sh.nb / W));
    const int64_t off = t * sh.n_kv * sh.nb * 32 * es;
    const ReadSide k{static_cast<uint8_t *>(K) + off, bias, kp}, v{static_cast<uint8_t *>(V) + off, nullptr, vp};
    const dim3 grid((n_items + kThreads / 4 - 1) / (kThreads / 4), 2);
    err = by_types(kt, vt, elem, [&](auto k_, auto v_, auto e_) {
      auto go = [&](auto rot, auto w) {
        k_paged_read<k_.value, v_.value, e_.value, rot.value, w.value><<<grid, kThreads, 0, stream>>>(k, v, sh, slots + t, n_items, di->err_word);
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

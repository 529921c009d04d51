// norm.cu — root-mean-square norm of rows with the residual's addition and an
// output in Q8_0 blocks (include/bq.h: bq_add_rms_norm).
//
//   h = x + r rounded to the rows' type;  rstd = fl32(1 / sqrt(sum h^2 / n + eps));
//   y = fl32(fl32(h rstd) w);  outputs: h, y rounded to the rows' type, y in Q8_0.
//
// The 8-bit codes hang on the last bit of rstd, and every quantizer here is
// exact to the bit, so rstd is too: the sum of squares is carried as an
// unevaluated sum of two floats (each square's rounding error by one fused
// multiply-add, each addition's by Knuth's two-sum), relative error about 2^-44
// in any order of the lanes, and 1 / sqrt by one Newton step whose residual is
// computed in the same form. The rounded factor then differs from that of the
// exact sum with a probability around 2^-19 per row. (Doubles would give the
// same, at 1/64 of the rate: 4096 of them per row take longer than the row's
// memory time.)
//
// Bound by HBM and, with 16-bit rows, by how fast few warps issue (at 6000 x 4096, 59 %
// of the active cycles with 4 warps a scheduler, DRAM 46 %): a row stays in
// registers from its load to its last output, values go through in pairs (packed
// fp32 instructions), and the 34-byte blocks are put together in shared memory,
// from where they leave in 16-byte stores. 16384 bf16 rows of 4096 with all outputs
// (608 MB): 110 us, 5.5 TB/s; fp32 rows to Q8_0 (876 MB) 162 us, 5.4 TB/s; one row
// to sixteen of 4096: 3.4 us.
#include <algorithm>

#include "bq_device.cuh"
#include "bq_internal.h"
#include "layer.h"
#include "paged.cuh"

namespace bq {
namespace {

// An unevaluated sum of two floats, |l| <= half a step of h.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.h, b.h);
  const float l = __fadd_rn(s.l, __fadd_rn(a.l, b.l)), h = __fadd_rn(s.h, l);
  return Two{h, __fsub_rn(l, __fsub_rn(h, s.h))};
}
// without the last normalization: the low parts stay small enough for some twenty such sums
__device__ __forceinline__ Two add_loose(Two a, Two b) {
  const Two s = two_sum(a.h, b.h);
  return Two{s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l))};
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  const float p = __fmul_rn(a.h, b.h);
  const float e = __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.h, b.h, -p)));
  const float h = __fadd_rn(p, e);
  return Two{h, __fsub_rn(e, __fsub_rn(h, p))};
}

// fl32(1 / sqrt(s / n + eps)) of a sum of squares
__device__ __forceinline__ float factor(Two s, const NormArgs &a) {
  const Two m = add(mul(s, Two{a.inv_n[0], a.inv_n[1]}), Two{a.eps[0], a.eps[1]});
  const float r = rsqrtf(m.h);
  // 1 - m r^2, the terms of r^2 and of the product each with their errors
  const float r2 = __fmul_rn(r, r), r2l = __fmaf_rn(r, r, -r2);
  const float p = __fmul_rn(m.h, r2);
  const float pl = __fmaf_rn(m.l, r2, __fmaf_rn(m.h, r2l, __fmaf_rn(m.h, r2, -p)));
  return __fmaf_rn(r, 0.5f * __fsub_rn(__fsub_rn(1.0f, p), pl), r);
}

// Two such sums at once
struct Two2 {
  uint64_t h, l;
};
__device__ __forceinline__ uint64_t two(float x) { return pack2(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ float lo(uint64_t v) { return __uint_as_float(uint32_t(v)); }
__device__ __forceinline__ float hi(uint64_t v) { return __uint_as_float(uint32_t(v >> 32)); }
__device__ __forceinline__ uint64_t fsub2(uint64_t a, uint64_t b) { return ffma2(two(-1.0f), b, a); }

// 8 values of a row as they lie in memory, and as pairs
template <int ELEM>
struct Raw8 {
  uint4 w[ELEM == kElemF32 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t *p) {
    w[0] = __ldcs(reinterpret_cast<const uint4 *>(p));
    if constexpr (ELEM == kElemF32) w[1] = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
  }
  __device__ __forceinline__ void zero() {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (ELEM == kElemF32) w[1] = w[0];
  }
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    if constexpr (ELEM == kElemF32) {
      v[0] = pack2(w[0].x, w[0].y), v[1] = pack2(w[0].z, w[0].w), v[2] = pack2(w[1].x, w[1].y), v[3] = pack2(w[1].z, w[1].w);
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_pair<ELEM>(u[i]);
        v[i] = pack2(__float_as_uint(f.x), __float_as_uint(f.y));
      }
    }
  }
};
template <int ELEM>
__device__ __forceinline__ void store8(uint8_t *p, const uint64_t (&v)[4]) {
  if constexpr (ELEM == kElemF32) {
    *reinterpret_cast<float4 *>(p) = make_float4(lo(v[0]), hi(v[0]), lo(v[1]), hi(v[1]));
    *(reinterpret_cast<float4 *>(p) + 1) = make_float4(lo(v[2]), hi(v[2]), lo(v[3]), hi(v[3]));
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_pair<ELEM>(lo(v[0]), hi(v[0])), pack_pair<ELEM>(lo(v[1]), hi(v[1])),
                                               pack_pair<ELEM>(lo(v[2]), hi(v[2])), pack_pair<ELEM>(lo(v[3]), hi(v[3])));
  }
}

// m / 127 rounded once, for the magnitudes whose quotient is not far below
// binary16's range (the others round to a scale of zero either way): a quotient
// within one step, its exact remainder, and the correction by the correctly rounded
// reciprocal, which gives the rounded quotient (Markstein 1990, theorem 7; the
// divisor's significand is not all ones).
__device__ __forceinline__ float div127(float m) {
  const float y = 1.0f / 127.0f, q = __fmul_rn(m, y);
  return __fmaf_rn(__fmaf_rn(-127.0f, q, m), y, q);
}

// 8 codes as two words of bytes: the rule of quantize_block_lane, exact per value
__device__ __forceinline__ void codes8(const uint64_t (&v)[4], float ds, float inv, uint32_t &w0, uint32_t &w1) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  uint32_t t[8];
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t r = fmul2(v[i], two(inv)), q = fadd2(r, two(kMagic)), e = fsub2(r, fadd2(q, two(-kMagic)));
    t[2 * i] = uint32_t(q);
    t[2 * i + 1] = uint32_t(q >> 32);
    far = fmaxf(far, fmaxf(fabsf(lo(e)), fabsf(hi(e))));
  }
  if (far > 0.4999f || (ds > 0.0f && ds < 6.103515625e-05f)) {  // rare: near a tie, or a subnormal scale
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[2 * i] = uint32_t(code_of<kTypeQ8_0>(lo(v[i]), ds, inv));
      t[2 * i + 1] = uint32_t(code_of<kTypeQ8_0>(hi(v[i]), ds, inv));
    }
  }
  w0 = pack_bytes(t[0], t[1], t[2], t[3]);
  w1 = pack_bytes(t[4], t[5], t[6], t[7]);
}

// Rows by blockDim.x threads each, blockDim.y of them at a time in a CTA (more than
// one only where a warp has a row), the next ones' loads in flight while these are
// worked on; a thread has U units of 8 values, 4 lanes a block.
template <int ELEM, int U, int MAX>
__global__ void __launch_bounds__(MAX, U == 4 ? 512 / MAX : MAX == 256 ? 3 : MAX == 128 ? 6 : 1) k_add_rms_norm(const NormArgs a) {
  __shared__ Two part[2][32];
  extern __shared__ __align__(16) uint8_t staged[];  // the rows' blocks, each row as far past 16 bytes as in q8
  constexpr int ES = Elem<ELEM>::kBytes;
  const int n_units = a.n_cols / 8, step = blockDim.x, lane = threadIdx.x & 31;
  const int row_bytes = a.n_cols / kQK * Fmt<kTypeQ8_0>::kBytes;
  const bool words = row_bytes % 4 == 0;  // an even number of blocks: rows of whole words
  const int64_t stride = int64_t(gridDim.x) * blockDim.y;
  Raw8<ELEM> x[U], r[U];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = threadIdx.x + u * step;
      if (unit < n_units) {
        x[u].load(a.x + row * a.x_row + int64_t(unit) * 8 * ES);
        if (a.res) r[u].load(a.res + row * a.res_row + int64_t(unit) * 8 * ES);
      }
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) x[u].zero(), r[u].zero();
  int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row < a.n_rows) fetch(row);
  // rows end for whole warps; with several warps per row there is one row per CTA
  for (int turn = 0; row < a.n_rows; row += stride, turn ^= 1) {
    uint64_t v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = threadIdx.x + u * step;
      x[u].get(v[u]);
      if (a.res && unit < n_units) {
        uint64_t w[4];
        r[u].get(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = fadd2(v[u][i], w[i]);
        uint8_t *to = a.sum + row * a.sum_row + int64_t(unit) * 8 * ES;
        if constexpr (ELEM == kElemF32) {
          if (a.sum) store8<ELEM>(to, v[u]);
        } else {
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[i] = pack_pair<ELEM>(lo(v[u][i]), hi(v[u][i]));
            const float2 f = unpack_pair<ELEM>(h[i]);
            v[u][i] = pack2(__float_as_uint(f.x), __float_as_uint(f.y));
          }
          if (a.sum) *reinterpret_cast<uint4 *>(to) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
    }
    if (row + stride < a.n_rows) fetch(row + stride);
    Two2 s2{0, 0};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t p = fmul2(v[u][i], v[u][i]);
        const uint64_t sum = fadd2(s2.h, p), t = fsub2(sum, s2.h);
        uint64_t e = fadd2(fsub2(s2.h, fsub2(sum, t)), fsub2(p, t));
        // a 16-bit type's square has no error (22 bits at most)
        if constexpr (ELEM == kElemF32) e = fadd2(e, ffma2(v[u][i], v[u][i], fsub2(0, p)));
        s2 = Two2{sum, fadd2(s2.l, e)};
      }
    Two s = add_loose(Two{lo(s2.h), lo(s2.l)}, Two{hi(s2.h), hi(s2.l)});
#pragma unroll
    for (int d = 16; d; d >>= 1) s = add_loose(s, Two{__shfl_xor_sync(kFull, s.h, d), __shfl_xor_sync(kFull, s.l, d)});
    if (step > 32) {
      const int warp = threadIdx.x >> 5, warps = step >> 5;
      if (lane == 0) part[turn][warp] = s;
      __syncthreads();
      s = lane < warps ? part[turn][lane] : Two{0.0f, 0.0f};
      for (int d = warps <= 4 ? 2 : warps <= 8 ? 4 : 16; d; d >>= 1) s = add_loose(s, Two{__shfl_xor_sync(kFull, s.h, d), __shfl_xor_sync(kFull, s.l, d)});
      if (warps <= 8) s = Two{__shfl_sync(kFull, s.h, 0), __shfl_sync(kFull, s.l, 0)};
    } else {
      __syncwarp();  // the row before this one has left the staging place
    }
    const float f = factor(add(s, Two{0.0f, 0.0f}), a);
    uint8_t *const q8 = a.q8 + row * row_bytes;
    const int shift = words ? int(reinterpret_cast<uintptr_t>(q8) & 15) : 0;
    uint8_t *const stage = staged + threadIdx.y * ((row_bytes + 32) / 16 * 16) + shift;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = threadIdx.x + u * step;
      const bool live = unit < n_units;  // the same for the 4 lanes of a block, and with words for those of two
      float m = 0.0f;
      if (live) {
        const float4 w0 = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * unit), w1 = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * unit + 1);
        const uint64_t w[4] = {pack2(__float_as_uint(w0.x), __float_as_uint(w0.y)), pack2(__float_as_uint(w0.z), __float_as_uint(w0.w)),
                               pack2(__float_as_uint(w1.x), __float_as_uint(w1.y)), pack2(__float_as_uint(w1.z), __float_as_uint(w1.w))};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[u][i] = fmul2(fmul2(v[u][i], two(f)), w[i]);
          m = fmaxf(m, fmaxf(fabsf(lo(v[u][i])), fabsf(hi(v[u][i]))));
        }
        if (a.out) store8<ELEM>(a.out + row * a.out_row + int64_t(unit) * 8 * ES, v[u]);
      }
      if (a.q8) {
        m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
        m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
        const uint16_t bits = __half_as_ushort(__float2half_rn(div127(m)));
        const float ds = half_bits_to_float(bits);
        uint32_t w0, w1;
        codes8(v[u], ds, ds > 0.0f ? rcp_approx(ds) : 0.0f, w0, w1);
        if (words) {
          // two blocks are 17 words: those of the first lie two bytes off its codes
          const uint32_t before = __shfl_up_sync(kFull, w1 >> 16, 1);
          const int j = unit & 7;
          if (live) {
            uint32_t *pair = reinterpret_cast<uint32_t *>(stage + unit / 8 * 68);
            const bool first = j < 4;
            const int at = 2 * j + !first;
            pair[at] = first ? (j == 0 ? bits : before) | w0 << 16 : w0;
            pair[at + 1] = first ? __funnelshift_r(w0, w1, 16) : w1;
            if (j == 4) pair[8] = before | uint32_t(bits) << 16;
          }
        } else if (live) {
          uint16_t *block = reinterpret_cast<uint16_t *>(q8 + unit / 4 * Fmt<kTypeQ8_0>::kBytes);
          const int j = unit & 3;
          if (j == 0) block[0] = bits;
          block[1 + 4 * j] = uint16_t(w0);
          block[2 + 4 * j] = uint16_t(w0 >> 16);
          block[3 + 4 * j] = uint16_t(w1);
          block[4 + 4 * j] = uint16_t(w1 >> 16);
        }
      }
    }
    if (a.q8 && words) {
      if (step > 32)
        __syncthreads();
      else
        __syncwarp();
      const uint8_t *from = stage - shift;
      uint8_t *to = q8 - shift;
      for (int i = threadIdx.x * 16; i < shift + row_bytes; i += step * 16) {
        if (i >= shift && i + 16 <= shift + row_bytes) {
          *reinterpret_cast<uint4 *>(to + i) = *reinterpret_cast<const uint4 *>(from + i);
        } else {
          for (int k = i; k < i + 16; k += 4)
            if (k >= shift && k < shift + row_bytes) *reinterpret_cast<uint32_t *>(to + k) = *reinterpret_cast<const uint32_t *>(from + k);
        }
      }
    }
  }
}

template <int ELEM, int U, int MAX>
cudaError_t launch(const NormArgs &a, int threads, int rows, int sms, cudaStream_t stream) {
  const int row_bytes = a.n_cols / kQK * Fmt<kTypeQ8_0>::kBytes;
  const int smem = a.q8 && row_bytes % 4 == 0 ? rows * ((row_bytes + 32) / 16 * 16) : 0;
  const void *fn = reinterpret_cast<const void *>(k_add_rms_norm<ELEM, U, MAX>);
  cudaError_t e = ensure_smem(fn, smem);
  if (e != cudaSuccess) return e;
  int64_t grid = (a.n_rows + rows - 1) / rows;
  if (grid > sms) {  // as many CTAs as are resident, each with rows to come
    int per_sm = 0;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, threads * rows, smem)) != cudaSuccess) return e;
    grid = std::min(grid, int64_t(sms) * std::max(per_sm, 1));
  }
  k_add_rms_norm<ELEM, U, MAX><<<unsigned(grid), dim3(threads, rows), smem, stream>>>(a);
  return cudaGetLastError();
}

template <int ELEM>
cudaError_t launch_elem(const NormArgs &a, int sms, cudaStream_t stream) {
  const int units = a.n_cols / 8;
  auto threads = [&](int u) { return (units + 32 * u - 1) / (32 * u) * 32; };  // whole warps, u units each
  if (units <= 32) return launch<ELEM, 1, 128>(a, 32, 4, sms, stream);
  // few rows: a row's latency counts, so one unit per thread
  if (a.n_rows <= 2 * sms && threads(1) <= 1024) return launch<ELEM, 1, 1024>(a, threads(1), 1, sms, stream);
  if (units <= 64) return launch<ELEM, 2, 128>(a, 32, 4, sms, stream);
  if (units <= 128) return launch<ELEM, 4, 128>(a, 32, 4, sms, stream);
  // four units where three warps or more have a row: the sums over its threads are
  // a quarter of the instructions then, half with two (112 us for 115 at 16384 x 4096)
  if (units <= 256) return launch<ELEM, 2, 256>(a, threads(2), 1, sms, stream);
  if (units <= 512) return launch<ELEM, 4, 128>(a, threads(4), 1, sms, stream);
  if (units <= 1024) return launch<ELEM, 4, 256>(a, threads(4), 1, sms, stream);
  if (units <= 2048) return launch<ELEM, 2, 1024>(a, threads(2), 1, sms, stream);
  return launch<ELEM, 8, 1024>(a, 1024, 1, sms, stream);
}

}  // namespace

cudaError_t launch_add_rms_norm(int elem, const NormArgs &a, cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  if (elem == kElemF32) return launch_elem<kElemF32>(a, di->sm_count, stream);
  if (elem == kElemF16) return launch_elem<kElemF16>(a, di->sm_count, stream);
  return launch_elem<kElemBF16>(a, di->sm_count, stream);
}

}  // namespace bq

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

// 8 values of a row as fp32
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
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
template <int ELEM>
__device__ __forceinline__ void store8(uint8_t *p, const float (&v)[8]) {
  if constexpr (ELEM == kElemF32) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *(reinterpret_cast<float4 *>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_pair<ELEM>(v[0], v[1]), pack_pair<ELEM>(v[2], v[3]),
                                               pack_pair<ELEM>(v[4], v[5]), pack_pair<ELEM>(v[6], v[7]));
  }
}
// rounded to the rows' type
template <int ELEM>
__device__ __forceinline__ void round8(float (&v)[8]) {
  if constexpr (ELEM != kElemF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_pair<ELEM>(pack_pair<ELEM>(v[2 * i], v[2 * i + 1]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}

// A row by blockDim.x threads, blockDim.y rows per CTA (more than one only
// where a warp has a row); a thread has U units of 8 values, 4 lanes a block.
template <int ELEM, int U>
__global__ void __launch_bounds__(1024) k_add_rms_norm(const NormArgs a) {
  __shared__ Two part[32];
  constexpr int ES = Elem<ELEM>::kBytes;
  const int n_units = a.n_cols / 8, step = blockDim.x;
  const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= a.n_rows) return;  // whole warps; with several warps per row there is one row per CTA
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int unit = threadIdx.x + u * step;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
    if (unit < n_units) load8<ELEM>(a.x + row * a.x_row + int64_t(unit) * 8 * ES, v[u]);
  }
  if (a.res) {
    float r[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = threadIdx.x + u * step;
      if (unit < n_units) load8<ELEM>(a.res + row * a.res_row + int64_t(unit) * 8 * ES, r[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = threadIdx.x + u * step;
      if (unit < n_units) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = __fadd_rn(v[u][i], r[u][i]);
        round8<ELEM>(v[u]);
        if (a.sum) store8<ELEM>(a.sum + row * a.sum_row + int64_t(unit) * 8 * ES, v[u]);
      }
    }
  }
  Two s{0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = __fmul_rn(v[u][i], v[u][i]);
      const Two t = two_sum(s.h, p);
      // a 16-bit type's square has no error (22 bits at most)
      s = Two{t.h, __fadd_rn(s.l, ELEM == kElemF32 ? __fadd_rn(t.l, __fmaf_rn(v[u][i], v[u][i], -p)) : t.l)};
    }
  s = add(s, Two{0.0f, 0.0f});
#pragma unroll
  for (int d = 16; d; d >>= 1) s = add(s, Two{__shfl_xor_sync(kFull, s.h, d), __shfl_xor_sync(kFull, s.l, d)});
  if (step > 32) {
    const int warp = threadIdx.x >> 5, warps = step >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = s;
    __syncthreads();
    s = part[0];
    for (int w = 1; w < warps; ++w) s = add(s, part[w]);
  }
  const float f = factor(s, a);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int unit = threadIdx.x + u * step;
    const bool live = unit < n_units;  // the same for the 4 lanes of a block
    float m = 0.0f;
    if (live) {
      const float4 w0 = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * unit), w1 = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * unit + 1);
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[u][i] = __fmul_rn(__fmul_rn(v[u][i], f), w[i]);
        m = fmaxf(m, fabsf(v[u][i]));
      }
      if (a.out) store8<ELEM>(a.out + row * a.out_row + int64_t(unit) * 8 * ES, v[u]);
    }
    if (a.q8) {
      m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
      m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
      if (live) {
        uint16_t bits;
        float ds;
        block_scale<kTypeQ8_0>(m, bits, ds);
        const float inv = ds > 0.0f ? rcp_approx(ds) : 0.0f;
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = uint32_t(code_of<kTypeQ8_0>(v[u][i], ds, inv));
        uint16_t *block = reinterpret_cast<uint16_t *>(a.q8 + (row * (a.n_cols / kQK) + unit / 4) * Fmt<kTypeQ8_0>::kBytes);
        const int j = unit & 3;
        if (j == 0) block[0] = bits;
#pragma unroll
        for (int i = 0; i < 4; ++i) block[1 + 4 * j + i] = uint16_t((c[2 * i] & 255) | (c[2 * i + 1] << 8));
      }
    }
  }
}

template <int ELEM, int U>
cudaError_t launch(const NormArgs &a, int threads, int rows, cudaStream_t stream) {
  k_add_rms_norm<ELEM, U><<<unsigned((a.n_rows + rows - 1) / rows), dim3(threads, rows), 0, stream>>>(a);
  return cudaGetLastError();
}

template <int ELEM>
cudaError_t launch_elem(const NormArgs &a, cudaStream_t stream) {
  const int units = a.n_cols / 8;
  if (units <= 32) return launch<ELEM, 1>(a, 32, 4, stream);
  if (units <= 128) return launch<ELEM, 4>(a, 32, 4, stream);
  const int t4 = (units + 127) / 128 * 32;  // threads for 4 units each, whole warps
  if (t4 <= 1024) return launch<ELEM, 4>(a, t4, 1, stream);
  return launch<ELEM, 8>(a, 1024, 1, stream);
}

}  // namespace

cudaError_t launch_add_rms_norm(int elem, const NormArgs &a, cudaStream_t stream) {
  if (elem == kElemF32) return launch_elem<kElemF32>(a, stream);
  if (elem == kElemF16) return launch_elem<kElemF16>(a, stream);
  return launch_elem<kElemBF16>(a, stream);
}

}  // namespace bq

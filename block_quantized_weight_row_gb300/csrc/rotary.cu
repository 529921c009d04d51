// rotary.cu — rotary positions on several axes (include/bq.h: bq_rotary).
//
// Pair i of a head's first `rot` channels is turned by pos[axis[i]][t] * f_i:
//   (a, b) -> (a cos - b sin, a sin + b cos).
//
// The angle is kept as a 64-bit fraction of a turn: with F_i = f_i / 2 pi mod 1
// as a multiple of 2^-64, pos * F_i modulo 2^64 (one integer product) is the
// turn's fraction, off by at most |pos| 2^-54 of a turn from the double F_i was
// made of, for any position. Its upper half, signed, is an angle in [-1/2, 1/2)
// turns, exact to 2^-33, for sincospif, which needs no range reduction: a far
// position costs and errs no more than a near one (fp32 angles lose all digits
// from positions around 2^24 on).
//
// Bound by HBM: q and k are read and written once. A CTA makes the sines and
// cosines of a few tokens once, in shared memory, for all heads of both tensors.
#include <algorithm>

#include "bq_device.cuh"
#include "bq_internal.h"
#include "layer.h"
#include "paged.cuh"

namespace bq {
namespace {

template <int ELEM>
__device__ __forceinline__ float load1(const uint8_t *p) {
  if constexpr (ELEM == kElemF32) return *reinterpret_cast<const float *>(p);
  if constexpr (ELEM == kElemF16) return __half2float(*reinterpret_cast<const __half *>(p));
  if constexpr (ELEM == kElemBF16) return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p));
}
template <int ELEM>
__device__ __forceinline__ void store1(uint8_t *p, float v) {
  if constexpr (ELEM == kElemF32) *reinterpret_cast<float *>(p) = v;
  if constexpr (ELEM == kElemF16) *reinterpret_cast<__half *>(p) = __float2half_rn(v);
  if constexpr (ELEM == kElemBF16) *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(v);
}

// frequency -> 2^64ths of a turn per position
__device__ __forceinline__ uint64_t turns(double f) {
  const double t = f * 0.15915494309189533577;
  const double frac = t - floor(t);  // [0, 1]
  return uint64_t(__double2ull_rz(frac * 4294967296.0)) << 32 |
         uint64_t(__double2uint_rz((frac * 4294967296.0 - floor(frac * 4294967296.0)) * 4294967296.0));
}

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // of a CTA

template <int IN, int OUT>
__global__ void __launch_bounds__(kThreads) k_rotary(const RotaryArgs a) {
  extern __shared__ float2 cs[];  // [token][pair]
  constexpr int IS = Elem<IN>::kBytes, OS = Elem<OUT>::kBytes;
  const int pairs = a.rot / 2;
  const int64_t t0 = int64_t(blockIdx.x) * kTokens;
  const int nt = int(min(int64_t(kTokens), a.n_tokens - t0));
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int tt = i / pairs, p = i - tt * pairs;
    int ax = a.axis ? a.axis[p] : 0;
    if (uint32_t(ax) >= uint32_t(a.n_axes)) {
      atomicOr(a.err, kErrIndex);
      ax = 0;
    }
    const int64_t pos = a.pos[ax * a.pos_axis + t0 + tt];
    const uint64_t turn = uint64_t(pos) * turns(a.inv_freq[p]);
    float s, c;
    sincospif(float(int32_t((turn + 0x80000000u) >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: halves of a turn
    cs[i] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();
  const int rest = a.in_place ? 0 : a.dim - a.rot;
  const int items = pairs + rest, heads = a.heads[0] + a.heads[1];
  for (int i = threadIdx.x; i < nt * heads * items; i += kThreads) {
    const int r = i / items, p = i - r * items;
    const int tt = r / heads;
    int h = r - tt * heads;
    const bool k = h >= a.heads[0];
    if (k) h -= a.heads[0];
    const RotarySide &s = a.side[k];
    const uint8_t *in = s.in + (t0 + tt) * s.in_token + h * s.in_head;
    uint8_t *out = s.out + (t0 + tt) * s.out_token + h * s.out_head;
    if (p < pairs) {
      const int ca = a.interleaved ? 2 * p : p, cb = a.interleaved ? 2 * p + 1 : p + pairs;
      const float x = load1<IN>(in + ca * IS), y = load1<IN>(in + cb * IS);
      const float2 w = cs[tt * pairs + p];
      store1<OUT>(out + ca * OS, __fmaf_rn(x, w.x, -__fmul_rn(y, w.y)));
      store1<OUT>(out + cb * OS, __fmaf_rn(x, w.y, __fmul_rn(y, w.x)));
    } else {
      const int c = a.rot + p - pairs;
      store1<OUT>(out + c * OS, load1<IN>(in + c * IS));
    }
  }
}

template <int IN, int OUT>
cudaError_t launch(const RotaryArgs &a, cudaStream_t stream) {
  const int smem = kTokens * (a.rot / 2) * 8;
  cudaError_t e = ensure_smem(reinterpret_cast<const void *>(k_rotary<IN, OUT>), smem);
  if (e != cudaSuccess) return e;
  k_rotary<IN, OUT><<<unsigned((a.n_tokens + kTokens - 1) / kTokens), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(int elem_in, int elem_out, RotaryArgs a, cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  a.err = di->err_word;
  if (elem_in == kElemF32 && elem_out == kElemF32) return launch<kElemF32, kElemF32>(a, stream);
  if (elem_in == kElemF32 && elem_out == kElemF16) return launch<kElemF32, kElemF16>(a, stream);
  if (elem_in == kElemF32) return launch<kElemF32, kElemBF16>(a, stream);
  if (elem_in == kElemF16) return launch<kElemF16, kElemF16>(a, stream);
  return launch<kElemBF16, kElemBF16>(a, stream);
}

}  // namespace bq

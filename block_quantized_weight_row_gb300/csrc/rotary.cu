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
// cosines of a few tokens once, in shared memory, for all heads of both tensors;
// then its threads take units of 16 bytes of output, four at a time, loads first.
// A unit's partner channels are in the unit (adjacent pairs), in another one that
// the same thread takes (halves of a multiple of the unit), or are gathered (other
// halves: each lane loads them beside its own unit, from L1).
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
  const double t = f * 0.15915494309189533577;  // 1 / 2 pi
  return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// V channels as fp32
template <int ELEM, int V>
__device__ __forceinline__ void load(const uint8_t *p, float (&v)[V]) {
  if constexpr (ELEM == kElemF32) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 f = *(reinterpret_cast<const float4 *>(p) + i);
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
  } else {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_pair<ELEM>(u[i]);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
template <int ELEM, int V>
__device__ __forceinline__ void store(uint8_t *p, const float (&v)[V]) {
  if constexpr (ELEM == kElemF32)
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_pair<ELEM>(v[0], v[1]), pack_pair<ELEM>(v[2], v[3]), pack_pair<ELEM>(v[4], v[5]), pack_pair<ELEM>(v[6], v[7]));
}

__device__ __forceinline__ float2 turn_pair(float x, float y, float2 w) {
  return make_float2(__fmaf_rn(x, w.x, -__fmul_rn(y, w.y)), __fmaf_rn(x, w.y, __fmul_rn(y, w.x)));
}

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // of a CTA

// How a unit finds its partners
enum Path { kAdjacent, kHalves, kGather, kScalar };

// units: of a head (with kHalves, a unit of the first half stands for both); tokens: of a CTA
template <int IN, int OUT, int PATH>
__global__ void __launch_bounds__(kThreads) k_rotary(const RotaryArgs a, const int units, const int tokens) {
  constexpr int IS = Elem<IN>::kBytes, OS = Elem<OUT>::kBytes;
  constexpr int V = PATH == kScalar ? 1 : 16 / OS;        // channels of a unit
  constexpr int P = PATH == kAdjacent ? V / 2 : V;        // pairs of a unit
  constexpr int NB = PATH == kGather || PATH == kScalar ? 1 : PATH == kHalves ? 2 : 4;  // units in flight
  extern __shared__ uint64_t freq[];  // per pair, then cosine and sine per token and pair
  const int pairs = a.rot / 2;
  const int cols = (pairs + P - 1) / P;  // pair p of a token at (p % P) * cols + p / P: neighbouring units meet no bank twice
  float2 *const table = reinterpret_cast<float2 *>(freq + pairs);
  const int64_t t0 = int64_t(blockIdx.x) * tokens;
  const int nt = int(min(int64_t(tokens), a.n_tokens - t0));
  for (int p = threadIdx.x; p < pairs; p += kThreads) freq[p] = turns(a.inv_freq[p]);
  __syncthreads();
  for (int i = threadIdx.x; i < nt * cols * P; i += kThreads) {
    const int tt = i / (cols * P), p = i - tt * (cols * P);
    float s = 0.0f, c = 1.0f;  // beyond the last pair channels stay as they are
    if (p < pairs) {
      int ax = a.axis ? __ldg(a.axis + p) : 0;
      if (uint32_t(ax) >= uint32_t(a.n_axes)) {
        atomicOr(a.err, kErrIndex);
        ax = 0;
      }
      const uint64_t turn = uint64_t(int64_t(__ldg(a.pos + ax * a.pos_axis + t0 + tt))) * freq[p];
      sincospif(float(int32_t((turn + 0x80000000u) >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: halves of a turn
    }
    table[tt * cols * P + (p % P) * cols + p / P] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();
  const int heads = a.heads[0] + a.heads[1], n = nt * heads * units;
  for (int i0 = threadIdx.x; i0 < n; i0 += NB * kThreads) {
    float x[NB][PATH == kHalves ? 2 : 1][V];
    const uint8_t *in[NB];
    uint8_t *out[NB];
    int unit[NB], tok[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int i = i0 + b * kThreads;
      unit[b] = -1;
      if (i < n) {
        const int r = i / units, tt = r / heads;
        unit[b] = i - r * units;
        tok[b] = tt;
        int h = r - tt * heads;
        const bool k = h >= a.heads[0];
        if (k) h -= a.heads[0];
        const RotarySide &s = a.side[k];
        in[b] = s.in + (t0 + tt) * s.in_token + h * s.in_head;
        out[b] = s.out + (t0 + tt) * s.out_token + h * s.out_head;
        if constexpr (PATH == kAdjacent || PATH == kGather) load<IN, V>(in[b] + unit[b] * V * IS, x[b][0]);
        if constexpr (PATH == kHalves) {
          // a unit of the first half with its partner, or two of the channels behind
          const int c = unit[b] < cols ? unit[b] * V : a.rot + 2 * (unit[b] - cols) * V;
          load<IN, V>(in[b] + c * IS, x[b][0]);
          load<IN, V>(in[b] + (c + (unit[b] < cols ? pairs : V)) * IS, x[b][1]);
        }
      }
    }
    if constexpr (PATH == kAdjacent || PATH == kHalves) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (unit[b] >= 0) {
          const bool turned = unit[b] < cols;
          const float2 *w = table + tok[b] * cols * P + unit[b];
          if (turned) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
              float &u = PATH == kHalves ? x[b][0][j] : x[b][0][2 * j], &v = PATH == kHalves ? x[b][PATH == kHalves][j] : x[b][0][2 * j + 1];
              const float2 f = turn_pair(u, v, w[j * cols]);
              u = f.x, v = f.y;
            }
          }
          if constexpr (PATH == kAdjacent) {
            store<OUT, V>(out[b] + unit[b] * V * OS, x[b][0]);
          } else {
            const int c = turned ? unit[b] * V : a.rot + 2 * (unit[b] - cols) * V;
            store<OUT, V>(out[b] + c * OS, x[b][0]);
            store<OUT, V>(out[b] + (c + (turned ? pairs : V)) * OS, x[b][PATH == kHalves]);
          }
        }
    } else if constexpr (PATH == kGather) {
      // a head is `units` lanes of one warp (units a power of two up to 32): all load before one stores
      if (unit[0] >= 0) {
        const float2 *w = table + tok[0] * cols * P;
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = unit[0] * V + j;
          y[j] = c < a.rot ? load1<IN>(in[0] + (c < pairs ? c + pairs : c - pairs) * IS) : 0.0f;
        }
        __syncwarp((units == 32 ? kFull : (1u << units) - 1) << (threadIdx.x & 31 & ~(units - 1)));
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = unit[0] * V + j, p = c < pairs ? c : c - pairs;
          if (c < a.rot) {
            const float2 f = w[(p % P) * cols + p / P];
            x[0][0][j] = c < pairs ? __fmaf_rn(x[0][0][j], f.x, -__fmul_rn(y[j], f.y)) : __fmaf_rn(y[j], f.y, __fmul_rn(x[0][0][j], f.x));
          }
        }
        store<OUT, V>(out[0] + unit[0] * V * OS, x[0][0]);
      }
    } else {
      const int p = unit[0];  // a pair, then the channels behind
      if (p < pairs) {
        const float2 f = turn_pair(load1<IN>(in[0] + p * IS), load1<IN>(in[0] + (p + pairs) * IS), table[tok[0] * cols + p]);
        store1<OUT>(out[0] + p * OS, f.x);
        store1<OUT>(out[0] + (p + pairs) * OS, f.y);
      } else {
        const int c = p + pairs;
        store1<OUT>(out[0] + c * OS, load1<IN>(in[0] + c * IS));
      }
    }
  }
}

template <int IN, int OUT, int PATH>
cudaError_t launch_path(const RotaryArgs &a, int sms, cudaStream_t stream) {
  constexpr int V = PATH == kScalar ? 1 : 16 / Elem<OUT>::kBytes, P = PATH == kAdjacent ? V / 2 : V;
  const int pairs = a.rot / 2, cols = (pairs + P - 1) / P;
  // in place, the units that no pair reaches need nothing
  const int units = PATH == kAdjacent ? (a.in_place ? cols : a.dim / V)
                  : PATH == kHalves   ? (a.in_place ? cols : a.dim / (2 * V))
                  : PATH == kGather   ? a.dim / V
                                      : (a.in_place ? pairs : a.dim - pairs);
  // tokens of a CTA: enough units for four of each thread, where CTAs remain for four waves
  const int64_t work = int64_t(units) * (a.heads[0] + a.heads[1]);
  int tokens = 1;
  while (tokens < kMaxTokens && tokens * work < 4 * kThreads && a.n_tokens / (2 * tokens) >= int64_t(sms) * 16) tokens *= 2;
  while (tokens > 1 && (pairs + tokens * cols * P) * 8 > 100 * 1024) tokens /= 2;
  const int smem = (pairs + tokens * cols * P) * 8;
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(k_rotary<IN, OUT, PATH>), smem);
  if (e != cudaSuccess) return e;
  k_rotary<IN, OUT, PATH><<<unsigned((a.n_tokens + tokens - 1) / tokens), kThreads, smem, stream>>>(a, units, tokens);
  return cudaGetLastError();
}

template <int IN, int OUT>
cudaError_t launch(const RotaryArgs &a, int sms, cudaStream_t stream) {
  constexpr int V = 16 / Elem<OUT>::kBytes;
  const int units = a.dim / V;
  if (a.interleaved) return launch_path<IN, OUT, kAdjacent>(a, sms, stream);
  if (a.rot / 2 % V == 0) return launch_path<IN, OUT, kHalves>(a, sms, stream);
  if (units <= 32 && (units & (units - 1)) == 0) return launch_path<IN, OUT, kGather>(a, sms, stream);
  return launch_path<IN, OUT, kScalar>(a, sms, stream);
}

}  // namespace

cudaError_t launch_rotary(int elem_in, int elem_out, RotaryArgs a, cudaStream_t stream) {
  cudaError_t err;
  const DeviceInfo *di = device_info(&err);
  if (!di) return err;
  a.err = di->err_word;
  if (elem_in == kElemF32 && elem_out == kElemF32) return launch<kElemF32, kElemF32>(a, di->sm_count, stream);
  if (elem_in == kElemF32 && elem_out == kElemF16) return launch<kElemF32, kElemF16>(a, di->sm_count, stream);
  if (elem_in == kElemF32) return launch<kElemF32, kElemBF16>(a, di->sm_count, stream);
  if (elem_in == kElemF16) return launch<kElemF16, kElemF16>(a, di->sm_count, stream);
  return launch<kElemBF16, kElemBF16>(a, di->sm_count, stream);
}

}  // namespace bq

// rotary.cu — rotary positions on several axes (include/bq.h: bq_rotary).
//
// Pair i of a head's first `rot` channels is turned by pos[axis[i]][t] * f_i:
//   (a, b) -> (a cos - b sin, a sin + b cos).
//
// The angle is kept as a 64-bit fraction of a turn: with F_i = f_i / 2 pi mod 1
// as a multiple of 2^-64, pos * F_i modulo 2^64 (one integer product) is the
// turn's fraction, off by at most |pos| (2^-52 |f_i| / 2 pi + 2^-54) of a turn from the
// double F_i was made of, for any position. Its upper half, signed, is an angle in
// [-1/2, 1/2) turns, exact to 2^-33: its upper 24 bits, which fp32 holds, go to
// sincospif, which needs no range reduction, and the lower 8 turn the result on by
// their small angle (as one float the angle was off by up to 2^-26 of a turn). A far
// position costs and errs no more than a near one (fp32 angles lose all digits
// from positions around 2^24 on).
//
// Bound by HBM: q and k are read and written once. A CTA makes the sines and
// cosines of a few tokens once, in shared memory, for all heads of both tensors;
// then its threads take units of 16 bytes of output, several at a time, loads
// first, the first of them before the sines; a CTA has as many tokens as make the
// grid one wave. 32768 tokens of 32 + 8 bf16 heads of 128 (671 MB): 117 us, 5.7 TB/s
// (pair by pair, with an integer division each, 365 us); 32 tokens 3 us.
// A unit's partner channels are in the unit (adjacent pairs), in another one that
// the same thread takes (halves of a multiple of the unit), or are gathered (other
// halves: each lane loads them beside its own unit, from L1; onto the input itself
// where a head fits a warp's lanes, else pair by pair).
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

// V channels as they lie in memory, and as fp32
template <int ELEM, int V>
struct Raw {
  static constexpr int kWords = V * Elem<ELEM>::kBytes / 16;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const uint8_t *p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = *(reinterpret_cast<const uint4 *>(p) + i);
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (ELEM == kElemF32) {
          v[4 * i + k] = __uint_as_float(u[k]);
        } else {
          const float2 f = unpack_pair<ELEM>(u[k]);
          v[2 * k] = f.x, v[2 * k + 1] = f.y;
        }
      }
    }
  }
};
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
constexpr int kMaxTokens = 32;  // of a CTA
constexpr int kResident = 4;     // CTAs of an SM (64 registers)

// How a unit finds its partners
enum Path { kAdjacent, kHalves, kGather, kScalar };

// units: of a head (with kHalves, a unit of the first half stands for both); tokens: of a CTA
template <int IN, int OUT, int PATH>
__global__ void __launch_bounds__(kThreads, kResident) k_rotary(const RotaryArgs a, const int units, const int tokens) {
  constexpr int IS = Elem<IN>::kBytes, OS = Elem<OUT>::kBytes;
  constexpr int V = PATH == kScalar ? 1 : 16 / OS;   // channels of a unit
  constexpr int P = PATH == kAdjacent ? V / 2 : V;   // pairs of a unit
  constexpr int W = PATH == kHalves ? 2 : 1;         // units that are turned together
  constexpr bool kWide = PATH == kAdjacent || PATH == kHalves;
  constexpr int NB = !kWide ? 1 : 4 / (W * (IS / OS));  // in flight
  constexpr int LV = PATH == kScalar ? 16 / IS : V;  // (the scalar path keeps none)
  extern __shared__ uint64_t freq[];  // per pair, then cosine and sine per token and pair
  const int pairs = a.rot / 2;
  const int cols = (pairs + P - 1) / P;  // pair p of a token at (p % P) * cols + p / P: neighbouring units meet no bank twice
  float2 *const table = reinterpret_cast<float2 *>(freq + pairs);
  const int64_t t0 = int64_t(blockIdx.x) * tokens;
  const int nt = int(min(int64_t(tokens), a.n_tokens - t0));
  const int heads = a.heads[0] + a.heads[1], n = nt * heads * units;

  // item i: a unit of a head of a token, and where its head lies
  struct Item {
    const uint8_t *in;
    uint8_t *out;
    int unit, tok;  // unit < 0: none
  };
  auto item = [&](int i) {
    Item x{nullptr, nullptr, -1, 0};
    if (i < n) {
      const int r = i / units;
      x.unit = i - r * units;
      x.tok = r / heads;
      int h = r - x.tok * heads;
      const bool k = h >= a.heads[0];
      if (k) h -= a.heads[0];
      const RotarySide &s = a.side[k];
      x.in = s.in + (t0 + x.tok) * s.in_token + h * s.in_head;
      x.out = s.out + (t0 + x.tok) * s.out_token + h * s.out_head;
    }
    return x;
  };
  // with kHalves: a unit of the first half and its partner, or two of the channels behind
  auto channel = [&](int unit, int k) {
    if constexpr (PATH == kHalves) return unit < cols ? unit * V + k * pairs : a.rot + (2 * (unit - cols) + k) * V;
    return unit * V;
  };
  Item it[NB];
  Raw<IN, LV> x[NB][W];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      it[b] = item(i0 + b * kThreads);
      if constexpr (PATH != kScalar)
        if (it[b].unit >= 0) {
#pragma unroll
          for (int k = 0; k < W; ++k) x[b][k].load(it[b].in + channel(it[b].unit, k) * IS);
        }
    }
  };
  fetch(threadIdx.x);

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
      const int32_t angle = int32_t((turn + 0x80000000u) >> 32), low = angle & 255;
      sincospif(float(angle - low) * 4.656612873077393e-10f, &s, &c);  // 2^-31: halves of a turn
      const float d = float(low) * 1.4629180792671596e-9f, s0 = s;     // pi 2^-31; up to 3.8e-7, so that 1 - cos d, 7e-14, is nothing
      s = __fmaf_rn(d, c, s);
      c = __fmaf_rn(-d, s0, c);
    }
    table[tt * cols * P + (p % P) * cols + p / P] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();

  for (int i0 = threadIdx.x; i0 < n;) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (it[b].unit < 0) continue;
      const int unit = it[b].unit;
      const float2 *w = table + it[b].tok * cols * P;
      if constexpr (kWide) {
        float v[W][V];
#pragma unroll
        for (int k = 0; k < W; ++k) x[b][k].get(v[k]);
        if (unit < cols) {
#pragma unroll
          for (int j = 0; j < P; ++j) {
            // a unit that reaches past `rot`: its other channels as they are (a turn by 0 would make inf - inf of an infinity beside)
            if (PATH == kAdjacent && unit * P + j >= pairs) continue;
            float &u = PATH == kHalves ? v[0][j] : v[0][2 * j], &y = PATH == kHalves ? v[W - 1][j] : v[0][2 * j + 1];
            const float2 f = turn_pair(u, y, w[j * cols + unit]);
            u = f.x, y = f.y;
          }
        }
#pragma unroll
        for (int k = 0; k < W; ++k) store<OUT, V>(it[b].out + channel(unit, k) * OS, v[k]);
      } else if constexpr (PATH == kGather) {
        // onto the input itself a head is `units` lanes of one warp (a power of two up to 32): all load before one stores
        float v[V], y[V];
        x[b][0].get(v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = unit * V + j;
          y[j] = c < a.rot ? load1<IN>(it[b].in + (c < pairs ? c + pairs : c - pairs) * IS) : 0.0f;
        }
        if (a.onto) __syncwarp((units == 32 ? kFull : (1u << units) - 1) << (threadIdx.x & 31 & ~(units - 1)));
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = unit * V + j, p = c < pairs ? c : c - pairs;
          if (c < a.rot) {
            const float2 f = w[(p % P) * cols + p / P];
            v[j] = c < pairs ? __fmaf_rn(v[j], f.x, -__fmul_rn(y[j], f.y)) : __fmaf_rn(y[j], f.y, __fmul_rn(v[j], f.x));
          }
        }
        store<OUT, V>(it[b].out + unit * V * OS, v);
      } else if (unit < pairs) {  // a pair, then the channels behind
        const float2 f = turn_pair(load1<IN>(it[b].in + unit * IS), load1<IN>(it[b].in + (unit + pairs) * IS), w[unit]);
        store1<OUT>(it[b].out + unit * OS, f.x);
        store1<OUT>(it[b].out + (unit + pairs) * OS, f.y);
      } else {
        const int c = unit + pairs;
        store1<OUT>(it[b].out + c * OS, load1<IN>(it[b].in + c * IS));
      }
    }
    i0 += NB * kThreads;
    if (i0 < n) fetch(i0);
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
  int tokens = int(std::min<int64_t>(kMaxTokens, (a.n_tokens + int64_t(sms) * kResident - 1) / (int64_t(sms) * kResident)));
  while (tokens > 1 && (pairs + tokens * cols * P) * 8 > 48 * 1024) tokens /= 2;
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
  if (!a.onto || (units <= 32 && (units & (units - 1)) == 0)) return launch_path<IN, OUT, kGather>(a, sms, stream);
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

// lora.cuh — what the two files of the adapters' kernels share: a tile's tokens,
// the sums of a cluster, launches (lora.cu has the mathematics and the plan).
#pragma once

#include <cooperative_groups.h>

#include "bq_device.cuh"
#include "bq_internal.h"
#include "layer.h"
#include "paged.cuh"
#include "tcgen05.cuh"

namespace bq {

constexpr int kLeaders = 256;  // up to this many tokens, CTAs find their tiles themselves
constexpr int kMaxBins = 4096 + 1;  // adapters, and the tokens without one

struct LoraTile {
  int adapter, first, count, unused;  // first: in the sorted tokens
};

// Workspace: H, then (grouped) the sorted tokens, the tiles and their number.
struct LoraWork {
  float *H;         // [token][rank]
  int32_t *sorted;  // null: tiles by leaders
  LoraTile *tiles;
  int32_t *n_tiles;
};

__device__ __forceinline__ int adapter_of(const LoraArgs &a, int t) {
  const int id = __ldg(a.adapter + t);
  return uint32_t(id) < uint32_t(a.n_adapters) ? id : -1;
}

// The tokens of tile `index` into rows[] (those beyond the count repeat the
// first), by all threads of the CTA. False: there is no such tile.
template <int TM>
__device__ __forceinline__ bool find_tile(const LoraArgs &a, const LoraWork &w, int index, int *rows, int &adapter, int &count) {
  __shared__ int before[8], total[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (w.sorted) {
    if (index >= *w.n_tiles) return false;
    const LoraTile t = w.tiles[index];
    adapter = t.adapter;
    count = t.count;
    if (tid < TM) rows[tid] = w.sorted[t.first + (tid < t.count ? tid : 0)];
    __syncthreads();
    return true;
  }
  // tokens of the adapter of token `index`, in order: with two passes of 128
  // threads or one of 256, every warp has whole groups of 32 tokens
  adapter = adapter_of(a, index);
  if (tid < 8) before[tid] = 0;
  __syncthreads();
  for (int t = tid; t < kLeaders; t += blockDim.x) {
    const unsigned same = __ballot_sync(kFull, t < a.n_tokens && adapter_of(a, t) == adapter);
    if (lane == 0) before[t >> 5] = int(same);
  }
  __syncthreads();
  if (warp == 0) {  // words of matches -> ranks
    const unsigned word = lane < 8 ? unsigned(before[lane]) : 0u;
    int rank = __popc(word);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      const int o = __shfl_up_sync(kFull, rank, d);
      if (lane >= d) rank += o;
    }
    const int all = __shfl_sync(kFull, rank, 7);
    rank -= __popc(word);  // matches before this word
    const int mine = __shfl_sync(kFull, rank, index >> 5) +
                     __popc(__shfl_sync(kFull, word, index >> 5) & ((1u << (index & 31)) - 1));  // the leader's rank
    const int n = min(TM, all - mine);
    if (mine % TM == 0) {
      // lane i of 16 finds the token of rank mine + i
      if (lane < TM) rows[lane] = index;
      __syncwarp();
      if (lane < 8) {
        unsigned left = word;
        for (int r = rank; left; ++r, left &= left - 1)
          if (r >= mine && r < mine + TM) rows[r - mine] = lane * 32 + __ffs(left) - 1;
      }
    }
    if (lane == 0) total[0] = mine % TM == 0 ? n : 0;
  }
  __syncthreads();
  count = total[0];
  return count > 0;
}

// Two fp32 values cut to bf16, packed; the rests (exact) stay. Three such steps
// give all 24 bits of a value.
__device__ __forceinline__ uint32_t cut_pair(float &x, float &y) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  x = __fsub_rn(x, __uint_as_float(a & 0xffff0000u));
  y = __fsub_rn(y, __uint_as_float(b & 0xffff0000u));
  return __byte_perm(a, b, 0x7632);
}

// A cluster's sums of a tile: each of its CTAs adds up its share, over the CTAs
// and, in each, over PARTS pieces of k (kept `apart` floats from one another), in
// order. part: [token][rank] of every CTA, `pitch` floats per token, 16-byte aligned.
template <int PARTS>
__device__ __forceinline__ void sum_tile(const LoraArgs &a, const LoraWork &w, float *part, int pitch, int apart, const int *rows, int ad, int count, int first,
                                         int ranks, int split, int splits) {
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  cluster.sync();
  const float s = a.scale ? __ldg(a.scale + ad) : 1.0f;
  // the loads from all CTAs in flight together; four ranks at a time (they come in
  // eights) where a CTA has one piece, one at a time in the small tiles of four
  constexpr int V = PARTS == 1 ? 4 : 1;
  const int wide = ranks / V, n = count * wide;
  for (int e = split * blockDim.x + threadIdx.x; e < n; e += splits * blockDim.x) {
    const int row = e / wide, r = V * (e - row * wide);
    float v[8][PARTS][V];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < splits) {
        const float *p = cluster.map_shared_rank(part, c) + row * pitch + r;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          if constexpr (V == 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + q * apart);
            v[c][q][0] = f.x, v[c][q][1] = f.y, v[c][q][2] = f.z, v[c][q][3] = f.w;
          } else {
            v[c][q][0] = p[q * apart];
          }
        }
      }
    float sum[V] = {};
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < splits) {
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
          for (int k = 0; k < V; ++k) sum[k] += v[c][q][k];
      }
    float *to = w.H + int64_t(rows[row]) * a.rank + first + r;
    if constexpr (V == 4)
      *reinterpret_cast<float4 *>(to) = make_float4(sum[0] * s, sum[1] * s, sum[2] * s, sum[3] * s);
    else
      *to = sum[0] * s;
  }
  cluster.sync();  // the others' sums are read from here until now
}

__device__ __forceinline__ void copy16(void *to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// The power of two that brings a row of H to 2^14 .. 2^15, near the upper end of
// binary16, so that values down to 2^-17 of the largest keep the 22 bits of two terms
// (at 1 .. 2 those below 2^-3 of it lost some, and 2^-25 of it in all), within normal
// numbers; m: the lane's largest |value|. Its inverse goes to unscale[r].
__device__ __forceinline__ float scale_row(float m, float *unscale, int r, int lane) {
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
  const int e = min(max(int(__float_as_uint(m) >> 23), 16), 254);
  if (lane == 0) unscale[r] = __uint_as_float(uint32_t(e - 14) << 23);
  return __uint_as_float(uint32_t(268 - e) << 23);
}

struct LoraPlan {
  bool grouped;
  int tm, tiles, splits;  // tiles: at most as many; splits: set here for tiles of 16
  int64_t busy;
  size_t bytes;
  size_t sorted_off, tiles_off, n_off;
};

template <typename... P, typename... A>
cudaError_t launch_ex(void (*fn)(P...), dim3 grid, int threads, int smem, int cluster, bool dependent, cudaStream_t stream, A... args) {
  if (smem > 0) {
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(fn), smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[2];
  int n = 0;
  attr[n].id = cudaLaunchAttributeClusterDimension;
  attr[n].val.clusterDim.x = unsigned(cluster);
  attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
  ++n;
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// Tiles of 64 tokens on the tensor-memory kernels (lora_tc.cu); the first product not
// for fp32 rows beside fp16 adapters.
cudaError_t launch_lora_shrink_tc(int x_elem, int w_elem, const LoraArgs &a, const LoraWork &w, const LoraPlan &p, cudaStream_t s);
cudaError_t launch_lora_expand_tc(int w_elem, int y_elem, const LoraArgs &a, const LoraWork &w, const LoraPlan &p, int sms, cudaStream_t s);

}  // namespace bq

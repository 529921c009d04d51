// lora_tc.cu — the adapters' products for tiles of 64 tokens, on the fifth-
// generation tensor cores (lora.cu has the mathematics and the plan).
#include <algorithm>

#include "lora.cuh"

namespace bq {
namespace {

// ------------------------------------- expand on the tensor-memory kernel --

// Tiles of 64 tokens, 128 columns of out a turn: D[column][token] = B (128 x rank,
// straight from the adapter by TMA) times H's terms (64 tokens, operand made once
// per CTA) on tcgen05, accumulated over the terms in tensor memory. With columns
// as the accumulator's lanes, a warp's access to y and out is 32 neighbouring
// columns of one token: whole sectors at any alignment of the rows, and a 32 x 32
// piece costs 32 loads, 32 stores and one tensor-memory load. (The warp-level
// instructions above move the same piece with 350 instructions and 224 wavefronts
// of shared memory and L1, which bound them: 160 us for 8192 tokens of 11008
// columns at rank 64.)
// Warps 0-7: lanes 32 (w mod 4) .., tokens 32 (w / 4) .., in two steps of 16
// tokens, the next step's y in flight; warp 8: TMA; warp 9: MMA. All waits bounded.
constexpr int kTcThreads = 320, kTcCols = 128, kTcTokens = 64, kTcTmem = 2 * kTcTokens;
constexpr int kTcBTile = kTcCols * 128, kTcHTile = kTcTokens * 128;  // 64 ranks: rows of 128 bytes

struct ExpandTc {
  static constexpr int kStages = 3;  // of B: a block of 64 ranks each
  int blocks, terms;                 // blocks of 64 ranks
  __host__ __device__ int h_off() const { return kStages * kTcBTile; }
  __host__ __device__ int bar_off() const { return h_off() + terms * blocks * kTcHTile; }
  __host__ __device__ int bytes() const { return bar_off() + 128 + 1024; }  // + room to align the base
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// 16 consecutive columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Loads and stores under a predicate, without a branch (which would have each
// load waited for where its branch ends); the bits as they lie in memory.
__device__ __forceinline__ void load_if(bool live, const uint8_t *p, uint32_t &v) {
  asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n mov.b32 %0, 0;\n @q ld.global.cs.b32 %0, [%1];\n}\n" : "=&r"(v) : "l"(p), "r"(int(live)));
}
__device__ __forceinline__ void load16_if(bool live, const uint8_t *p, uint4 &v) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
      " @q ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"(int(live)));
}
__device__ __forceinline__ void load_half_if(bool live, const uint8_t *p, uint32_t &v) {
  asm volatile("{\n .reg .pred q;\n .reg .b16 h;\n setp.ne.b32 q, %2, 0;\n mov.b16 h, 0;\n @q ld.global.cs.b16 h, [%1];\n cvt.u32.u16 %0, h;\n}\n"
               : "=r"(v) : "l"(p), "r"(int(live)));
}
__device__ __forceinline__ void store_if(bool live, uint8_t *p, uint32_t v) {
  asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n @q st.global.cs.b32 [%0], %1;\n}\n" ::"l"(p), "r"(v), "r"(int(live)) : "memory");
}
__device__ __forceinline__ void store_half_if(bool live, uint8_t *p, uint32_t v) {
  asm volatile("{\n .reg .pred q;\n .reg .b16 h;\n setp.ne.b32 q, %2, 0;\n cvt.u16.u32 h, %1;\n @q st.global.cs.b16 [%0], h;\n}\n" ::"l"(p), "r"(v), "r"(int(live)) : "memory");
}

// The work of a grid is one run of turns, tile after tile, cut into equal pieces,
// one per CTA: a tile's preparation (its tokens, H's operand: 3 us) is then paid
// once or twice per CTA, and all CTAs end together.
template <int WE, int YE>
__global__ void __launch_bounds__(kTcThreads, 2)
    k_lora_expand_tc(const __grid_constant__ CUtensorMap bmap, const LoraArgs a, const LoraWork w, const ExpandTc e, const uint32_t spin) {
  extern __shared__ uint8_t raw[];
  __shared__ float unscale[kTcTokens];
  __shared__ int rows[kTcTokens];
  __shared__ __align__(16) int64_t y_off[kTcTokens], out_off[kTcTokens];
  __shared__ uint32_t tmem_slot;
  __shared__ int aborted;
  constexpr int kTerms = WE == kElemF16 ? 2 : YE == kElemF32 ? 3 : 2, YS = Elem<YE>::kBytes, S = ExpandTc::kStages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t *sm = raw + (((smem_u32(raw) + 1023u) & ~1023u) - smem_u32(raw));
  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + e.bar_off());
  uint64_t *b_full = bar, *b_empty = bar + 3, *d_full = bar + 6, *d_empty = bar + 8, *done = bar + 10;
  volatile int *abort_flag = &aborted;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 8);
    }
    mbar_init(done, 1);
    aborted = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(kTcTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  const int groups = (a.M + kTcCols - 1) / kTcCols;
  const int64_t units = int64_t(*w.n_tiles) * groups;
  const int64_t u1 = units * (blockIdx.x + 1) / gridDim.x;
  int done_turns = 0;  // with products, over all tiles: the barriers' phases
  int armed = 0;       // blocks of B that were asked for
  for (int64_t u = units * blockIdx.x / gridDim.x; u < u1;) {
    const int tile = int(u / groups), g0 = int(u - int64_t(tile) * groups), n_turns = int(min(u1 - u, int64_t(groups - g0)));
    u += n_turns;
    __syncthreads();  // the tile before this one is done with rows, offsets and H
    if (*abort_flag) break;
    int ad, count;
    if (!find_tile<kTcTokens>(a, w, tile, rows, ad, count)) break;
    if (ad < 0 && a.y == a.out) continue;
    if (tid < kTcTokens) {
      y_off[tid] = rows[tid] * a.y_row;
      out_off[tid] = rows[tid] * a.out_row;
    }
    // H's terms as the second operand: token rows of 64 ranks, 128-byte swizzled; a lane has two ranks
    if (ad >= 0) {
      for (int r = warp; r < kTcTokens; r += kTcThreads / 32) {
        float h[2][2], m = 0.0f;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int c = 64 * b + 2 * lane + i;
            h[b][i] = r < count && c < a.rank ? __ldcg(w.H + int64_t(rows[r]) * a.rank + c) : 0.0f;
            m = fmaxf(m, fabsf(h[b][i]));
          }
        float up = 1.0f;
        if constexpr (WE == kElemF16) up = scale_row(m, unscale, r, lane);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (b >= e.blocks) break;
          float x = h[b][0] * up, y = h[b][1] * up;
#pragma unroll
          for (int k = 0; k < kTerms; ++k) {
            const uint32_t v = pack_pair<WE>(x, y);
            const float2 f = unpack_pair<WE>(v);
            x -= f.x, y -= f.y;
            *reinterpret_cast<uint32_t *>(sm + e.h_off() + (k * e.blocks + b) * kTcHTile + sw128_off(r, lane >> 2) + (lane & 3) * 4) = v;
          }
        }
      }
      fence_async_smem();
    }
    __syncthreads();

    const int i0 = done_turns;  // turn i of the tile is turn i0 + i of the barriers
    if (ad >= 0) done_turns += n_turns;
    if (warp == 8) {
      if (lane == 0 && ad >= 0) {
        for (int q = i0 * e.blocks; q < (i0 + n_turns) * e.blocks; ++q) {  // block q of all turns
          const int st = q % S, turn = q / e.blocks - i0, b = q % e.blocks;
          if (!tc_wait(&b_empty[st], ((q / S) & 1) ^ 1, spin, abort_flag, a.err)) break;
          mbar_arrive_expect_tx(&b_full[st], uint32_t(kTcBTile));
          tma_load_3d(sm + st * kTcBTile, &bmap, b * 64, (g0 + turn) * kTcCols, ad, &b_full[st]);
          armed = q + 1;
        }
      }
    } else if (warp == 9) {
      if (lane == 0 && ad >= 0) {
        // kind::f16: fp32 accumulators, both operands of the adapters' type, K-major
        constexpr uint32_t kType = WE == kElemBF16 ? (1u << 7) | (1u << 10) : 0u;
        constexpr uint32_t kIdesc = (1u << 4) | kType | (uint32_t(kTcTokens >> 3) << 17) | (uint32_t(kTcCols >> 4) << 24);
        const uint32_t b0 = smem_u32(sm), h0 = smem_u32(sm + e.h_off());
        for (int i = i0; i < i0 + n_turns; ++i) {
          const int buf = i & 1;
          bool there = tc_wait(&d_empty[buf], ((i >> 1) & 1) ^ 1, spin, abort_flag, a.err);
          const uint32_t d = tmem + uint32_t(buf * kTcTokens);
          uint32_t more = 0;
          for (int b = 0; b < e.blocks && there; ++b) {
            const int q = i * e.blocks + b, st = q % S;
            there = tc_wait(&b_full[st], (q / S) & 1, spin, abort_flag, a.err);
            if (!there) break;
            tc_fence_after();
            const uint64_t b_desc = sw128_desc(b0 + st * kTcBTile);
            for (int k = kTerms - 1; k >= 0; --k) {
              const uint64_t h_desc = sw128_desc(h0 + (k * e.blocks + b) * kTcHTile);
              for (int n = 0; n < 4 && b * 64 + n * 16 < a.rank; ++n) {
                tc_mma(d, b_desc + uint64_t(2 * n), h_desc + uint64_t(2 * n), kIdesc, more);
                more = 1;
              }
            }
            tc_commit(&b_empty[st]);
          }
          if (!there) break;
          tc_commit(&d_full[buf]);
        }
      }
    } else {
      const int lg = warp & 3, t0 = (warp >> 2) * 32;
      const uint32_t lane_addr = tmem + (uint32_t(lg * 32) << 16);
      const int odd = lane & 1;
      // 16-bit rows, where their boundaries allow it: two columns of one token per access (188 us -> 125 for
      // 8192 tokens of 11008 columns, the predicated loads included; fp32 rows, whose 32 columns are a line of
      // 128 bytes, lose by it: 166 -> 184)
      const bool pairs = YS == 2 && a.y_vec && a.M % 2 == 0;
      // steps of 16 tokens: 2 per turn; the next one's y is asked for before this one's sums are.
      // The bits of y. With pairs: of the lane's and its neighbour's column of one token, the first of
      // two in the even lane, the second in the odd one (16-bit rows: one word); else of the lane's column
      uint32_t y[2][16];
      auto column = [&](int step) { return (g0 + (step >> 1)) * kTcCols + lg * 32 + lane; };
      auto ask = [&](int step, uint32_t (&v)[16]) {
        const int m = column(step), from = t0 + (step & 1) * 16, end = a.y && step < 2 * n_turns && m < a.M ? count : 0;
        if (pairs) {
          const uint8_t *p = a.y + int64_t(m - odd) * YS;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r = from + 2 * j + odd;
            load_if(r < end, p + y_off[r], v[j]);
          }
        } else {
          const uint8_t *p = a.y + int64_t(m) * YS;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int64_t o = y_off[from + j];
            if constexpr (YS == 4)
              load_if(from + j < end, p + o, v[j]);
            else
              load_half_if(from + j < end, p + o, v[j]);
          }
        }
      };
      bool ok = true;
      auto give = [&](int step, const uint32_t (&v)[16]) {
        const int turn = i0 + (step >> 1), m = column(step), from = t0 + (step & 1) * 16, end = m < a.M ? count : 0;
        uint32_t d[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) d[j] = 0;
        if (ad >= 0) {
          if ((step & 1) == 0) {
            ok = tc_wait_warp(&d_full[turn & 1], (turn >> 1) & 1, spin, abort_flag, a.err);
            if (!ok) return;
            tc_fence_after();
          }
          tmem_ld16(lane_addr + uint32_t((turn & 1) * kTcTokens + from), d);
          if (step & 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[turn & 1]);
          }
        }
        // the token's row of y plus its products; without an adapter y as it is
        auto sum = [&](uint32_t x, float with, int r) {
          return ad < 0 ? with : WE == kElemF16 ? __fmaf_rn(__uint_as_float(x), unscale[r], with) : __fadd_rn(__uint_as_float(x), with);
        };
        if (pairs) {
          uint8_t *p = a.out + int64_t(m - odd) * YS;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t other = __shfl_xor_sync(kFull, odd ? d[2 * j] : d[2 * j + 1], 1);
            const int r = from + 2 * j + odd;
            const uint32_t x0 = odd ? other : d[2 * j], x1 = odd ? d[2 * j + 1] : other;
            if constexpr (YS == 2) {
              const float2 with = unpack_pair<YE>(v[j]);
              store_if(r < end, p + out_off[r], pack_pair<YE>(sum(x0, with.x, r), sum(x1, with.y, r)));
            }
          }
        } else {
          uint8_t *p = a.out + int64_t(m) * YS;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int r = from + j;
            const int64_t o = out_off[r];
            if constexpr (YS == 4)
              store_if(r < end, p + o, __float_as_uint(sum(d[j], __uint_as_float(v[j]), r)));
            else
              store_half_if(r < end, p + o, pack_pair<YE>(sum(d[j], unpack_pair<YE>(v[j]).x, r), 0.0f));
          }
        }
      };
      ask(0, y[0]);
      for (int step = 0; step < 2 * n_turns && ok; step += 2) {
        ask(step + 1, y[1]);
        give(step, y[0]);
        if (!ok) break;
        ask(step + 2, y[0]);
        give(step + 1, y[1]);
      }
      tc_fence_before();
    }
  }
  // copies and products in flight end by themselves: none is left behind
  if (warp == 8 && lane == 0) {
    for (int i = 0; i < S && i < armed; ++i) {
      const int last = armed - 1 - ((armed - 1 - i) % S);
      tc_drain(&b_full[i], (last / S) & 1);
    }
  }
  if (warp == 9 && lane == 0) {
    tc_commit(done);
    tc_drain(done, 0);
  }
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcTmem) : "memory");
  }
}

// ------------------------------------- first product on tcgen05 --

// H of a tile of 64 tokens: D[rank][token] = A (up to 128 ranks x 64 k a stage,
// straight from the adapter by TMA; ranks it has not read as zeros) times the tokens'
// rows of x, in tensor memory. Rows go through registers, stages ahead, to where the
// operand's swizzle wants them; fp32 rows are cut into three bf16 terms, each an
// operand tile. K is cut over the CTAs of a cluster and, in a CTA, over four
// accumulators (256 columns), so that the products' chains stay short: four parts of
// k, or for fp32 rows two, each with the largest term apart from the others, whose
// instructions would cut its sum too (4096 rows of 8192 at rank 128: 1.1e-6 of the
// output's norm for 1.6e-6 with four parts); the sums of all meet in fp32 in a
// fixed order.
// For fp32 rows and for more than 64 ranks, where the warp-level kernel of lora.cu
// is slower: whole calls of 8192 tokens of 4096 to 11008 columns
// take 189 us for 219 (fp32, rank 64) and 216 for 231 (bf16, rank 128). Of the two CTAs
// of an SM each takes a stage in 1.6 us of fp32 rows (2.6 TB/s of x) and 1.2 us of 16-bit
// ones at rank 128, whatever the copies' form or depth.
// Warps 0-7: rows of x, then the sums; warp 8: TMA; warp 9: MMA. All waits bounded.
constexpr int kShThreads = 320, kShRegions = 4, kShTmem = kShRegions * kTcTokens;
constexpr int kShXTile = kTcTokens * 128, kShPitch = 128;

// ROWS: ranks of a stage, 64 or 128. With 64 the products still have 128 rows: those
// beyond, of what lies behind the tile, reach only sums that nobody reads.
template <int XE, int ROWS>
struct ShrinkTc {
  static constexpr int kTerms = XE == kElemF32 ? 3 : 1;
  static constexpr int kStages = XE == kElemF32 ? (ROWS == 64 ? 3 : 2) : (ROWS == 64 ? 6 : 4);
  static constexpr int kAhead = XE == kElemF32 ? 2 : 5;  // stages of x in registers
  static constexpr int kATile = ROWS * 128, kStage = kATile + kTerms * kShXTile;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kBytes = kBarOff + 256 + 1024;  // + room to align the base
  static_assert(kStage >= 128 * 128, "the last stage's products stay inside");
  static_assert(kBarOff >= kTcTokens * kShPitch * 4, "the sums' place");
};

template <int XE, int WE, int ROWS>
__global__ void __launch_bounds__(kShThreads, 2)
    k_lora_shrink_tc(const __grid_constant__ CUtensorMap amap, const LoraArgs a, const LoraWork w, const int splits, const uint32_t spin) {
  using R = ShrinkTc<XE, ROWS>;
  constexpr int S = R::kStages, XS = Elem<XE>::kBytes;
  extern __shared__ uint8_t raw[];
  __shared__ int rows[kTcTokens];
  __shared__ uint32_t tmem_slot;
  __shared__ int aborted;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  int ad, count;
  if (!find_tile<kTcTokens>(a, w, blockIdx.y, rows, ad, count) || ad < 0) return;  // all CTAs of the cluster alike
  uint8_t *sm = raw + (((smem_u32(raw) + 1023u) & ~1023u) - smem_u32(raw));
  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + R::kBarOff);
  uint64_t *a_full = bar, *x_full = bar + S, *empty = bar + 2 * S, *done = bar + 3 * S;
  volatile int *abort_flag = &aborted;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&a_full[i], 1);
      mbar_init(&x_full[i], 8);
      mbar_init(&empty[i], 1);
    }
    mbar_init(done, 1);
    aborted = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(kShTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int split = blockIdx.x, all = (a.K + 63) / 64;
  const int s0 = int(int64_t(all) * split / splits), n = int(int64_t(all) * (split + 1) / splits) - s0;  // stages of 64 k
  constexpr int kParts = R::kTerms > 1 ? kShRegions / 2 : kShRegions;  // of k
  auto region = [&](int i) { return i * kParts / n; };
  float *part = reinterpret_cast<float *>(sm);

  if (warp < 8) {
    // a thread has 8 k (chunk c) of rows r and r + 32
    const int c = tid & 7, r = tid >> 3;
    const bool live[2] = {r < count, r + 32 < count};
    const uint8_t *src[2] = {a.x + rows[r] * a.x_row + (int64_t(s0) * 64 + c * 8) * XS, a.x + rows[r + 32] * a.x_row + (int64_t(s0) * 64 + c * 8) * XS};
    const uint32_t to[2] = {sw128_off(r, c), sw128_off(r + 32, c)};
    auto there = [&](int i) { return (s0 + i) * 64 + c * 8 < a.K; };
    bool ok = true;
    constexpr int kAhead = R::kAhead, kVec = XS / 2;  // stages in registers; 16-byte pieces of 8 k
    uint4 v[kAhead + 1][2][kVec];
    auto ask = [&](int i, uint4 (&q)[2][kVec]) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < kVec; ++k) load16_if(i < n && live[h] && there(i), src[h] + int64_t(i) * 64 * XS + 16 * k, q[h][k]);
    };
#pragma unroll
    for (int k = 0; k <= kAhead; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < kVec; ++q) v[k][h][q] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) ask(k, v[k]);
    // (buffers by constant indices: moving a register that a load is on its way to waits for it)
    for (int i0 = 0; i0 < n && ok; i0 += kAhead + 1)
#pragma unroll
    for (int u = 0; u <= kAhead; ++u) {
      const int i = i0 + u;
      if (i >= n) break;
      ask(i + kAhead, v[(u + kAhead) % (kAhead + 1)]);
      ok = tc_wait_warp(&empty[i % S], ((i / S) & 1) ^ 1, spin, abort_flag, a.err);
      if (!ok) break;
      uint8_t *x = sm + (i % S) * R::kStage + R::kATile;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (XE == kElemF32) {
          float f[8];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 q = v[u][h][k];
            f[4 * k] = __uint_as_float(q.x), f[4 * k + 1] = __uint_as_float(q.y), f[4 * k + 2] = __uint_as_float(q.z), f[4 * k + 3] = __uint_as_float(q.w);
          }
#pragma unroll
          for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint4 *>(x + k * kShXTile + to[h]) =
                make_uint4(cut_pair(f[0], f[1]), cut_pair(f[2], f[3]), cut_pair(f[4], f[5]), cut_pair(f[6], f[7]));
        } else {
          *reinterpret_cast<uint4 *>(x + to[h]) = v[u][h][0];
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x_full[i % S]);
    }
    // the sums of the four accumulators; the ring becomes their place once all products are done
    const int lg = warp & 3, half = warp >> 2;
    float acc[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = 0.0f;
    if (tc_wait_warp(done, 0, spin, abort_flag, a.err)) {
      tc_fence_after();
      for (int q = 0; q < kShRegions; ++q) {
        const int r = q * kParts / kShRegions, first = (r * n + kParts - 1) / kParts;  // the region's first stage, if it has one
        if (first >= n || region(first) != r) continue;
        uint32_t d[32];
        tmem_ld32(tmem + (uint32_t(lg * 32) << 16) + uint32_t(q * kTcTokens + half * 32), d);
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[j] += __uint_as_float(d[j]);
      }
      if (lg * 32 < a.rank) {
#pragma unroll
        for (int j = 0; j < 32; ++j) part[(half * 32 + j) * kShPitch + lg * 32 + lane] = acc[j];
      }
    }
    tc_fence_before();
  } else if (warp == 8) {
    if (lane == 0) {
      int armed = 0;
      for (int i = 0; i < n; ++i) {
        if (!tc_wait(&empty[i % S], ((i / S) & 1) ^ 1, spin, abort_flag, a.err)) break;
        mbar_arrive_expect_tx(&a_full[i % S], uint32_t(R::kATile));
        tma_load_3d(sm + (i % S) * R::kStage, &amap, (s0 + i) * 64, 0, ad, &a_full[i % S]);
        armed = i + 1;
      }
      for (int i = 0; i < S && i < armed; ++i) {  // never leave with a copy in flight
        const int last = armed - 1 - ((armed - 1 - i) % S);
        tc_drain(&a_full[i], (last / S) & 1);
      }
    }
  } else if (lane == 0) {
    constexpr uint32_t kType = WE == kElemBF16 ? (1u << 7) | (1u << 10) : 0u;
    constexpr uint32_t kIdesc = (1u << 4) | kType | (uint32_t(kTcTokens >> 3) << 17) | (uint32_t(128 >> 4) << 24);
    const uint32_t base = smem_u32(sm);
    int last = -1;  // region
    for (int i = 0; i < n; ++i) {
      const int st = i % S;
      if (!tc_wait(&a_full[st], (i / S) & 1, spin, abort_flag, a.err)) break;
      if (!tc_wait(&x_full[st], (i / S) & 1, spin, abort_flag, a.err)) break;
      tc_fence_after();
      const uint64_t a_desc = sw128_desc(base + st * R::kStage);
      const int steps = min(4, (a.K - (s0 + i) * 64) / 16);  // of 16 k
      const bool begun = region(i) == last;
      last = region(i);
      for (int k = R::kTerms - 1; k >= 0; --k) {
        const uint64_t x_desc = sw128_desc(base + st * R::kStage + R::kATile + k * kShXTile);
        const uint32_t d = tmem + uint32_t((R::kTerms > 1 ? 2 * last + (k > 0) : last) * kTcTokens);
        uint32_t more = begun || (k > 0 && k < R::kTerms - 1);
        for (int q = 0; q < steps; ++q) {
          tc_mma(d, a_desc + uint64_t(2 * q), x_desc + uint64_t(2 * q), kIdesc, more);
          more = 1;
        }
      }
      tc_commit(&empty[st]);
    }
    tc_commit(done);
    tc_drain(done, 0);
  }
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kShTmem) : "memory");
  }
  sum_tile<1>(a, w, part, kShPitch, 0, rows, ad, count, 0, a.rank, split, splits);
}

// [adapter][row][column] of 16-bit values in boxes of 64 columns (128 bytes,
// swizzled) x box_rows; columns and rows beyond an adapter's read as zeros
cudaError_t adapter_map(CUtensorMap &map, int w_elem, const uint8_t *base, int columns, int rows, int n, int box_rows) {
  map = CUtensorMap{};
  if (n == 0) return cudaSuccess;  // nobody loads from it
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encode();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {cuuint64_t(columns), cuuint64_t(rows), cuuint64_t(n)};
  const cuuint64_t strides[2] = {cuuint64_t(columns) * 2, cuuint64_t(columns) * 2 * cuuint64_t(rows)};
  const cuuint32_t box[3] = {64, cuuint32_t(box_rows), 1}, step[3] = {1, 1, 1};
  return encode(&map, w_elem == kElemBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint8_t *>(base), dims,
                strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int XE, int WE, int ROWS>
cudaError_t shrink64_rows(const LoraArgs &a, const LoraWork &w, const LoraPlan &p, cudaStream_t s) {
  CUtensorMap map;
  const cudaError_t e = adapter_map(map, WE, a.A, a.K, a.rank, a.n_adapters, ROWS);
  if (e != cudaSuccess) return e;
  return launch_ex(k_lora_shrink_tc<XE, WE, ROWS>, dim3(unsigned(p.splits), unsigned(p.tiles)), kShThreads, ShrinkTc<XE, ROWS>::kBytes, p.splits, true, s,
                   map, a, w, p.splits, spin_limit());
}
template <int XE, int WE>
cudaError_t shrink64(const LoraArgs &a, const LoraWork &w, const LoraPlan &p, cudaStream_t s) {
  return a.rank <= 64 ? shrink64_rows<XE, WE, 64>(a, w, p, s) : shrink64_rows<XE, WE, 128>(a, w, p, s);
}

template <int WE, int YE>
cudaError_t expand64(const LoraArgs &a, const LoraWork &w, const LoraPlan &p, int sms, cudaStream_t s) {
  CUtensorMap map;
  const cudaError_t st = adapter_map(map, WE, a.B, a.rank, a.M, a.n_adapters, kTcCols);
  if (st != cudaSuccess) return st;
  ExpandTc e;
  e.blocks = (a.rank + 63) / 64;
  e.terms = WE == kElemF16 ? 2 : YE == kElemF32 ? 3 : 2;
  const int64_t units = int64_t(p.tiles) * ((a.M + kTcCols - 1) / kTcCols);
  const int per_sm = e.bytes() <= 110 * 1024 ? 2 : 1;  // resident
  const dim3 grid(unsigned(std::min<int64_t>(units, int64_t(sms) * per_sm)));
  // not a dependent launch: CTAs that come while the first product's are still there
  // find less shared memory to share an SM, and the grid runs in two parts (200 us for 161)
  return launch_ex(k_lora_expand_tc<WE, YE>, grid, kTcThreads, e.bytes(), 1, false, s, map, a, w, e, spin_limit());
}

}  // namespace

cudaError_t launch_lora_shrink_tc(int x_elem, int w_elem, const LoraArgs &a, const LoraWork &w, const LoraPlan &p, cudaStream_t s) {
  if (w_elem == kElemF16) return shrink64<kElemF16, kElemF16>(a, w, p, s);
  return x_elem == kElemF32 ? shrink64<kElemF32, kElemBF16>(a, w, p, s) : shrink64<kElemBF16, kElemBF16>(a, w, p, s);
}

cudaError_t launch_lora_expand_tc(int w_elem, int y_elem, const LoraArgs &a, const LoraWork &w, const LoraPlan &p, int sms, cudaStream_t s) {
  if (w_elem == kElemBF16)
    return y_elem == kElemF32 ? expand64<kElemBF16, kElemF32>(a, w, p, sms, s) : expand64<kElemBF16, kElemBF16>(a, w, p, sms, s);
  return y_elem == kElemF32 ? expand64<kElemF16, kElemF32>(a, w, p, sms, s) : expand64<kElemF16, kElemF16>(a, w, p, sms, s);
}

}  // namespace bq

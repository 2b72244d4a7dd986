// Mixture-of-experts layer for a few tokens: every product of the chosen
// experts in two kernels, with the expert weights in FP8 and the activations
// at full precision.
//
//   gate/up kernel:  [g; u] = s13[e] * W13[e] x_t,  h = act(g) * u
//   down kernel:     y_t = sum_j w_tj * s2[e_j] * (W2[e_j] h_tj)
//
// Bound: the weights of the touched experts, read once from HBM (3 D F bytes
// an expert); a few tokens do 2 flops with each byte for each token.  So both
// kernels are one stream of weight tiles from HBM through TMA into shared
// memory and straight into tcgen05.mma, with no register in between.
//
// Weights are the M side of the MMA (128 rows of W), tokens the N side, which
// may be as narrow as 16 columns.  kind::f8f6f4 wants FP8 on both sides, so a
// token enters as the sum of two E4M3 vectors,
//   x * 2^(7-e) = hi + lo / 32,   2^e <= max |x| of the K slice < 2^(e+1),
// two columns of the MMA whose results the epilogue joins.  hi and lo keep 8
// significant bits: exact for BF16 activations down to 2^-15 of the slice's
// maximum (below that the error is under 2^-22 of the maximum), and for FP32
// ones no worse than a rounding to BF16.  A power of two as scale rounds
// nothing.  The scale belongs to one (token, K slice), and the epilogue adds
// the slices in FP32 registers.
//
// Roles of a CTA (persistent, one per SM):
//   warps 0-3   epilogue: TMEM lane quarter = warp; adds slices, applies the
//               expert's scale, activation or partial sums, joins tokens
//   warps 4-11  converters: read the tokens' K slice from L2, split it into
//               hi and lo, write the swizzled B tile (two buffers)
//   warp 12     producer: weight tiles of 128 rows x 128 K (16 KB) by TMA
//   warp 13     MMA issuer
// Work is cut into items (up to TT tokens of one expert) x (128 weight rows)
// x (K split); each CTA derives the list of items from the ids by itself, so
// no launch has to prepare it, and takes every grid-th item.
//
// The gate/up kernel's 128 rows are 64 gate rows and the 64 up rows that
// belong to them, so that h needs one exchange between warps and never goes
// to memory as g and u, unless K is split: then the parts of g and u are
// added, and the activation taken, where the down kernel reads them.
// The down kernel writes FP32 parts per (K split, pair); the CTA that brings
// a token's last part for a row block adds them in a fixed order, weights
// them and rounds once to BF16.  The result does not depend on which CTA
// that is.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fp8la {
namespace {

constexpr int kEpiWarps = 4;
constexpr int kConvWarps = 8;
constexpr int kProducerWarp = kEpiWarps + kConvWarps;
constexpr int kMmaWarp = kProducerWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int BM = 128;             // weight rows of an item
constexpr int BK = 128;             // K of a stage (bytes = FP8 values)
constexpr int kStageBytes = BM * BK;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTokens = 128;
constexpr int kMaxTopK = 16;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kMaxTiles = kMaxExperts + kMaxPairs / 16;
constexpr int kMaxSplit = 8;

// TT tokens of an item, KC stages of a K slice, STAGES of the weight ring.
template <int TT>
struct Cfg {
  static constexpr int KC = TT == 16 ? 4 : 2;
  static constexpr int STAGES = TT == 16 ? 10 : 8;
  static constexpr int kSlice = KC * BK;
  static constexpr int kLanes = kSlice / 16;      // converter lanes of a token
  static constexpr int kPass = 32 * kConvWarps / kLanes;  // tokens of a pass
  static constexpr int kPasses = TT / kPass;
  static constexpr int kChunkBytes = 2 * TT * BK;  // B tile of one stage
  static constexpr int kBBytes = KC * kChunkBytes;
  static constexpr int kTmemCols = 4 * TT;         // two buffers of 2 TT
  static constexpr int kRing = 0;
  static constexpr int kB = kRing + STAGES * kStageBytes;
  static constexpr int kXch = kB + 2 * kBBytes;    // up rows' sums, FP32
  static constexpr int kScale = kXch + TT * 64 * 4;
  static constexpr int kOrder = kScale + 4 * TT * 4;
  static constexpr int kTile = kOrder + kMaxPairs * 2;
  static constexpr int kTokParts = kTile + kMaxTiles * 8;
  static constexpr int kBar = kTokParts + kMaxTokens * 2;
  static constexpr int kNumBars = 2 * STAGES + 8;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kEnd = kMisc + 128;
  static constexpr int kAlloc = kEnd + 1024;
  static_assert(kPass * kPasses == TT, "passes");
  static_assert(kB % 1024 == 0 && kChunkBytes % 1024 == 0, "swizzle atoms");
  static_assert(kBar % 8 == 0, "mbarriers");
  static_assert(kThreads / 32 * kMaxExperts * 2 <= 2 * kBBytes,
                "the plan's counts overlay the B tiles");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

struct LayerArgs {
  const void *x;         // gate/up kernel
  int64_t ldx;
  int32_t x_bf16, x_vec;
  int32_t T, E, k, D, F;
  const int32_t *ids;
  const float *weights;
  const float *s13, *s2;
  float *h;              // [pairs][Fp], or with a split [S][pairs][2][Fp]
  int64_t Fp;
  float *part;           // [S][pairs][Dp]
  int64_t Dp;
  unsigned *counters;    // [T][row blocks of the down kernel]
  uint16_t *y;
  int64_t ldy;
  int32_t gelu;
  uint32_t fmt_bits;
  int32_t max_split;
  unsigned *status;
  uint64_t timeout_ns;
};

struct Tile {            // up to TT pairs of one expert
  uint16_t expert, first, count, pad;
};

// K split of `items` items of nk stages on `grid` CTAs: the fewest rounds of
// items, a stage's time for starting an item and for each further part that
// has to be added.  Both kernels and the host's sizes follow it.
__host__ __device__ __forceinline__ int choose_split(int64_t items, int nk,
                                                     int grid, int max_split) {
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int s = 1; s <= max_split && s <= nk; ++s) {
    const int64_t rounds = (items * s + grid - 1) / grid;
    const int64_t cost = rounds * ((nk + s - 1) / s + 1) + (s > 1 ? s : 0);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

// Two fp32 -> two E4M3 codes (lo in bits 0-7), round to nearest even.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 decode_e4m3x2(uint32_t c) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(c)));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h2));
}

// Loads 8 TMEM columns at each of two addresses and waits for both.
__device__ __forceinline__ void tmem_ld8_pair(uint32_t a0, uint32_t a1,
                                              float (&u)[8], float (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, "
      "[%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3]), "=f"(u[4]), "=f"(u[5]),
        "=f"(u[6]), "=f"(u[7]), "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]),
        "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
      : "r"(a0), "r"(a1)
      : "memory");
}

__device__ __forceinline__ float activate(float g, int gelu) {
  if (gelu) {
    const float t = tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g));
    return 0.5f * g * (1.0f + t);
  }
  return g / (1.0f + __expf(-g));
}

// The 16 elements from k on of one activation row (zeros at and past K).
__device__ __forceinline__ void load_row16(const void *x, int64_t row_off,
                                           int bf16, int vec, int k, int K,
                                           float (&v)[16]) {
  if (bf16) {
    const uint16_t *p = static_cast<const uint16_t *>(x) + row_off + k;
    if (vec && k + 16 <= K) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(p) + i);
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] = __uint_as_float(q[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(q[j] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = k + i < K ? __uint_as_float(static_cast<uint32_t>(__ldcg(p + i))
                                           << 16)
                         : 0.0f;
    }
    return;
  }
  const float *p = static_cast<const float *>(x) + row_off + k;
  if (vec && k + 16 <= K) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 w = __ldcg(reinterpret_cast<const float4 *>(p) + i);
      v[4 * i] = w.x;
      v[4 * i + 1] = w.y;
      v[4 * i + 2] = w.z;
      v[4 * i + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = k + i < K ? __ldcg(p + i) : 0.0f;
  }
}

// h of one pair, 16 elements from f on: as stored, or from the parts of g
// and u that a K split of the gate/up kernel left.
__device__ __forceinline__ void load_h16(const LayerArgs &a, int split, int pair,
                                         int f, float (&v)[16]) {
  if (split == 1) {
    load_row16(a.h, static_cast<int64_t>(pair) * a.Fp, 0, 1, f, a.F, v);
    return;
  }
  float u[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = u[i] = 0.0f;
  const int64_t pairs = static_cast<int64_t>(a.T) * a.k;
  for (int s = 0; s < split; ++s) {
    const int64_t row = (s * pairs + pair) * 2 * a.Fp;
    float t[16];
    load_row16(a.h, row, 0, 1, f, a.F, t);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += t[i];
    load_row16(a.h, row + a.Fp, 0, 1, f, a.F, t);
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] += t[i];
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = activate(v[i], a.gelu) * u[i];
}

template <int TT, bool UP>
__global__ void __launch_bounds__(kThreads, 1)
    moe_stage_kernel(const __grid_constant__ CUtensorMap tmW,
                     const LayerArgs a) {
  using C = Cfg<TT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *sbase = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  const uint32_t bar0 = base + C::kBar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto bready_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + b); };
  auto sdone_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 2 + b); };
  auto accfree_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 4 + b); };
  const uint32_t group_bar = bar0 + 8u * (2 * C::STAGES + 6);
  const uint32_t final_bar = bar0 + 8u * (2 * C::STAGES + 7);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sbase + C::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + C::kMisc + 4);
  int *warp_sums = reinterpret_cast<int *>(sbase + C::kMisc + 16);
  float *xch = reinterpret_cast<float *>(sbase + C::kXch);
  float *scales = reinterpret_cast<float *>(sbase + C::kScale);
  uint16_t *order = reinterpret_cast<uint16_t *>(sbase + C::kOrder);
  Tile *tile_list = reinterpret_cast<Tile *>(sbase + C::kTile);
  uint16_t *tok_parts = reinterpret_cast<uint16_t *>(sbase + C::kTokParts);
  uint16_t *by_warp = reinterpret_cast<uint16_t *>(sbase + C::kB);  // plan only

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bready_bar(b), kConvWarps);
      mbar_init(sdone_bar(b), 1);
      mbar_init(accfree_bar(b), kEpiWarps);
    }
    mbar_init(group_bar, kEpiWarps);
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  const int pairs = a.T * a.k;
  // Warps that share out the pairs in the plan, 32 at a time.
  const int groups = (pairs + 31) / 32;
  const int plan_warps = min(kThreads / 32, groups);
  for (int i = threadIdx.x; i < plan_warps * a.E; i += kThreads) by_warp[i] = 0;
  for (int t = threadIdx.x; t < kMaxTokens; t += kThreads) tok_parts[t] = 0;
  // The gate/up kernel waits here for what precedes the layer; the down
  // kernel may only start once all of the gate/up kernel's CTAs have passed
  // that point, so ids and weights are final for it too.
  if (UP) {
    pdl_wait();
    pdl_launch_dependents();
  }

  // ---------------------------------------------------------------- plan
  // The pairs of each expert in increasing order, in tiles of up to TT.  The
  // order has to be the same in every CTA, since the tiles of one expert may
  // be different CTAs' items; so places come from counts, not from atomics.
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  bool bad = false;
  const int g_lo = warp < plan_warps ? groups * warp / plan_warps : 0;
  const int g_hi = warp < plan_warps ? groups * (warp + 1) / plan_warps : 0;
  for (int gr = g_lo; gr < g_hi; ++gr) {
    const int p = 32 * gr + lane;
    int id = p < pairs ? __ldcg(a.ids + p) : -1;
    if (id < -1 || id >= a.E) {
      bad = true;
      id = -1;
    }
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    if (id >= 0 && (same & ((1u << lane) - 1u)) == 0)
      by_warp[warp * a.E + id] =
          static_cast<uint16_t>(by_warp[warp * a.E + id] + __popc(same));
    __syncwarp();
  }
  bad = __syncthreads_or(bad);
  constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
  int n_tiles;
  {
    // One scan for both: pairs in the low 16 bits, tiles in the high ones.
    int c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x * kPer + i;
      c[i] = 0;
      if (e < a.E)
        for (int w = 0; w < plan_warps; ++w) c[i] += by_warp[w * a.E + e];
      sum += c[i] | ((c[i] + TT - 1) / TT) << 16;
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int at = incl - sum, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int v = warp_sums[w];
      if (w < warp) at += v;
      all += v;
    }
    n_tiles = all >> 16;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x * kPer + i;
      if (e < a.E) {
        const int first = at & 0xffff;
        int t = at >> 16;
        for (int done = 0; done < c[i]; done += TT, ++t)
          tile_list[t] = {static_cast<uint16_t>(e),
                          static_cast<uint16_t>(first + done),
                          static_cast<uint16_t>(min(TT, c[i] - done)), 0};
        // From here on: where each warp's next pair of the expert goes.
        int next = first;
        for (int w = 0; w < plan_warps; ++w) {
          const int n = by_warp[w * a.E + e];
          by_warp[w * a.E + e] = static_cast<uint16_t>(next);
          next += n;
        }
      }
      at += c[i] | ((c[i] + TT - 1) / TT) << 16;
    }
    __syncthreads();
  }
  if (!bad) {
    for (int gr = g_lo; gr < g_hi; ++gr) {
      const int p = 32 * gr + lane;
      const int id = p < pairs ? __ldcg(a.ids + p) : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, id);
      const int rank = __popc(same & ((1u << lane) - 1u));
      if (id >= 0)
        order[by_warp[warp * a.E + id] + rank] = static_cast<uint16_t>(p);
      __syncwarp();
      if (id >= 0 && rank == 0)
        by_warp[warp * a.E + id] =
            static_cast<uint16_t>(by_warp[warp * a.E + id] + __popc(same));
      __syncwarp();
    }
    if (!UP) {
      for (int t = threadIdx.x; t < a.T; t += kThreads) {
        int n = 0;
        for (int j = 0; j < a.k; ++j) n += __ldcg(a.ids + t * a.k + j) >= 0;
        tok_parts[t] = static_cast<uint16_t>(n);
      }
    }
  } else {
    if (threadIdx.x == 0 && blockIdx.x == 0)
      atomicOr(a.status, kStatusBadDeviceArg);
    n_tiles = 0;
  }
  __syncthreads();

  const int grid = gridDim.x;
  const int K = UP ? a.D : a.F;
  const int rows = UP ? a.F : a.D;       // output rows (h or y)
  constexpr int kRows = UP ? BM / 2 : BM;
  const int nk = (K + BK - 1) / BK;
  const int rb = (rows + kRows - 1) / kRows;
  // The split of the gate/up kernel is needed by the down kernel too, and
  // the grids are the same.
  const int split_up = choose_split(
      static_cast<int64_t>(n_tiles) * ((a.F + BM / 2 - 1) / (BM / 2)),
      (a.D + BK - 1) / BK, grid, a.max_split);
  const int split =
      UP ? split_up
         : choose_split(static_cast<int64_t>(n_tiles) * rb, nk, grid, a.max_split);
  const int64_t items = static_cast<int64_t>(n_tiles) * rb * split;
  const uint32_t tmem_base = *tmem_slot;

  // Item i: the K split is innermost, then the tile (tiles of one expert are
  // neighbours, so its weights are still in L2 for the second), then rows.
  auto item = [&](int64_t i, Tile &t, int &r, int &sp, int &c0, int &c1) {
    sp = static_cast<int>(i % split);
    const int64_t q = i / split;
    t = tile_list[q % n_tiles];
    r = static_cast<int>(q / n_tiles);
    c0 = nk * sp / split;
    c1 = nk * (sp + 1) / split;
  };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t s = 0, ph = 0, issued = 0;
      bool ok = true;
      for (int64_t i = blockIdx.x; ok && i < items; i += grid) {
        Tile t;
        int r, sp, c0, c1;
        item(i, t, r, sp, c0, c1);
        for (int c = c0; c < c1; ++c) {
          if (!mbar_wait(empty_bar(s), ph ^ 1u, a.timeout_ns, a.status,
                         abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t dst = base + C::kRing + s * kStageBytes;
          mbar_arrive_expect_tx(full_bar(s), kStageBytes);
          if (UP) {
            tma_load_3d(dst, &tmW, full_bar(s), c * BK, r * kRows, t.expert);
            tma_load_3d(dst + kStageBytes / 2, &tmW, full_bar(s), c * BK,
                        a.F + r * kRows, t.expert);
          } else {
            tma_load_3d(dst, &tmW, full_bar(s), c * BK, r * kRows, t.expert);
          }
          ++issued;
          if (++s == C::STAGES) { s = 0; ph ^= 1u; }
        }
      }
      // Wait for the copies in flight before the CTA may exit.
      for (uint32_t st = 0; st < C::STAGES; ++st) {
        if (issued <= st) break;
        const uint32_t arms = (issued - 1 - st) / C::STAGES + 1;
        mbar_wait_drain(full_bar(st), (arms - 1) & 1u, a.timeout_ns, a.status);
      }
    }
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      uint32_t s = 0, ph = 0, g = 0;  // stage ring; slices so far
      bool ok = true;
      for (int64_t i = blockIdx.x; ok && i < items; i += grid) {
        Tile t;
        int r, sp, c0, c1;
        item(i, t, r, sp, c0, c1);
        const int npad = (t.count + 7) & ~7;
        const uint32_t idesc = idesc_e4m3_f32(BM, 2 * npad) | a.fmt_bits;
        for (int cs = c0; ok && cs < c1; cs += C::KC, ++g) {
          const uint32_t b = g & 1u, use = g >> 1;
          if (!mbar_wait(accfree_bar(b), (use & 1u) ^ 1u, a.timeout_ns,
                         a.status, abort_flag) ||
              !mbar_wait(bready_bar(b), use & 1u, a.timeout_ns, a.status,
                         abort_flag)) {
            ok = false;
            break;
          }
          const int ce = min(c1, cs + C::KC);
          for (int c = cs; c < ce; ++c) {
            if (!mbar_wait(full_bar(s), ph, a.timeout_ns, a.status,
                           abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t adesc =
                smem_desc_k128_sw128(base + C::kRing + s * kStageBytes);
            const uint64_t bdesc = smem_desc_k128_sw128(
                base + C::kB + b * C::kBBytes + (c - cs) * C::kChunkBytes);
#pragma unroll
            for (int q = 0; q < BK / 32; ++q)
              umma_f8f6f4(tmem_base + b * 2 * TT, adesc + 2u * q,
                          bdesc + 2u * q, idesc, (c > cs || q > 0) ? 1u : 0u);
            umma_commit(empty_bar(s));
            if (++s == C::STAGES) { s = 0; ph ^= 1u; }
          }
          if (ok) umma_commit(sdone_bar(b));
        }
      }
      umma_commit(final_bar);
      mbar_wait_drain(final_bar, 0, a.timeout_ns, a.status);
    }
  } else if (warp >= kEpiWarps) {
    // ---------------------------------------------------------- converters
    // h comes from the gate/up kernel; weights do not, so the producer of
    // the down kernel is already running.
    if (!UP) pdl_wait();
    const int ct = threadIdx.x - 32 * kEpiWarps;
    const int sub = ct % C::kLanes;    // 16 elements of the slice
    const int trow = ct / C::kLanes;   // token within a pass
    const uint32_t unit = static_cast<uint32_t>(sub & 7);
    uint32_t g = 0;
    bool ok = true;
    for (int64_t i = blockIdx.x; ok && i < items; i += grid) {
      Tile t;
      int r, sp, c0, c1;
      item(i, t, r, sp, c0, c1);
      const int npad = (t.count + 7) & ~7;
      for (int cs = c0; cs < c1; cs += C::KC, ++g) {
        const int kk = cs * BK + sub * 16;
        const bool in = cs + sub / 8 < c1;
        float v[C::kPasses][16];
#pragma unroll
        for (int p = 0; p < C::kPasses; ++p) {
          const int col = p * C::kPass + trow;
          if (p * C::kPass >= npad) break;
          if (in && col < t.count) {
            const int pair = order[t.first + col];
            if (UP)
              load_row16(a.x, static_cast<int64_t>(pair / a.k) * a.ldx, a.x_bf16,
                         a.x_vec, kk, K, v[p]);
            else
              load_h16(a, split_up, pair, kk, v[p]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[p][j] = 0.0f;
          }
        }
        const uint32_t b = g & 1u;
        const bool ready = mbar_wait(sdone_bar(b), ((g >> 1) & 1u) ^ 1u,
                                     a.timeout_ns, a.status, abort_flag);
        if (!__all_sync(0xffffffffu, ready)) {
          ok = false;
          break;
        }
        const uint32_t chunk =
            base + C::kB + b * C::kBBytes + (sub / 8) * C::kChunkBytes;
#pragma unroll
        for (int p = 0; p < C::kPasses; ++p) {
          const int col = p * C::kPass + trow;
          if (p * C::kPass >= npad) break;
          uint32_t top = 0;  // |x| as bits: NaN and infinity are the largest
#pragma unroll
          for (int j = 0; j < 16; ++j)
            top = max(top, __float_as_uint(v[p][j]) & 0x7fffffffu);
#pragma unroll
          for (int d = C::kLanes / 2; d > 0; d >>= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
          // A slice that holds an infinity or a NaN is multiplied by 0, which
          // makes those elements NaN, and with them every output of the token.
          const uint32_t eb = max(top >> 23, 8u);
          const float inv = eb == 255u ? 0.0f : __uint_as_float((261u - eb) << 23);
          if (sub == 0 && col < npad)
            scales[(g & 3u) * TT + col] =
                eb == 255u ? 1.0f : __uint_as_float((eb - 7u) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            hi[w] = lo[w] = 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float x0 = v[p][4 * w + 2 * q] * inv;
              const float x1 = v[p][4 * w + 2 * q + 1] * inv;
              const uint32_t c2 = cvt_e4m3x2(x0, x1);
              const float2 back = decode_e4m3x2(c2);
              hi[w] |= c2 << (16 * q);
              lo[w] |= cvt_e4m3x2((x0 - back.x) * 32.0f, (x1 - back.y) * 32.0f)
                       << (16 * q);
            }
          }
          // K-major rows of 128 bytes, 16-byte units swizzled by the row.
          if (in && col < npad) {
            const uint32_t rh = static_cast<uint32_t>(col);
            const uint32_t rl = static_cast<uint32_t>(npad + col);
            st_shared_v4(chunk + rh * BK + ((unit ^ (rh & 7u)) << 4), hi[0],
                         hi[1], hi[2], hi[3]);
            st_shared_v4(chunk + rl * BK + ((unit ^ (rl & 7u)) << 4), lo[0],
                         lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bready_bar(b));
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    if (!UP) pdl_wait();
    const int row = threadIdx.x;  // 0..127: TMEM lane = weight row of the item
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
    uint32_t gph = 0;
    // Barrier of the four warps, with a limit.
    auto group_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(group_bar);
      const bool ok = mbar_wait(group_bar, gph, a.timeout_ns, a.status, abort_flag);
      gph ^= 1u;
      return __all_sync(0xffffffffu, ok) != 0;
    };
    if (UP) {
      const int rb_down = (a.D + BM - 1) / BM;
      for (int i = blockIdx.x * 128 + row; i < a.T * rb_down; i += grid * 128)
        a.counters[i] = 0;
    } else if (!bad) {
      // Tokens without any expert.
      for (int t = blockIdx.x; t < a.T; t += grid)
        if (tok_parts[t] == 0)
          for (int d = row; d < a.D; d += 128) a.y[t * a.ldy + d] = 0;
    }
    uint32_t g = 0;
    bool ok = true;
    for (int64_t i = blockIdx.x; ok && i < items; i += grid) {
      Tile t;
      int r, sp, c0, c1;
      item(i, t, r, sp, c0, c1);
      const int npad = (t.count + 7) & ~7;
      float acc[TT];
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[j] = 0.0f;
      for (int cs = c0; cs < c1; cs += C::KC, ++g) {
        const uint32_t b = g & 1u;
        const bool ready = mbar_wait(sdone_bar(b), (g >> 1) & 1u, a.timeout_ns,
                                     a.status, abort_flag);
        if (!__all_sync(0xffffffffu, ready)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float *sc = scales + (g & 3u) * TT;
        const uint32_t col0 = lane_base + b * 2 * TT;
#pragma unroll
        for (int j = 0; j < TT / 8; ++j) {
          if (8 * j < npad) {
            float u[8], v[8];
            tmem_ld8_pair(col0 + 8 * j, col0 + npad + 8 * j, u, v);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              acc[8 * j + q] = fmaf(fmaf(v[q], 0.03125f, u[q]), sc[8 * j + q],
                                    acc[8 * j + q]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(accfree_bar(b));
      }
      if (!ok) break;
      const float ws = __ldg((UP ? a.s13 : a.s2) + t.expert);
      if (UP) {
        const int f = r * kRows + (row & 63);
        if (split > 1) {
          // Parts of g (rows 0-63) and u (rows 64-127).
          if (f < a.F) {
#pragma unroll
            for (int j = 0; j < TT; ++j)
              if (j < t.count)
                a.h[((static_cast<int64_t>(sp) * pairs + order[t.first + j]) * 2 +
                     (row >> 6)) * a.Fp + f] = acc[j] * ws;
          }
        } else {
          if (row >= 64) {
#pragma unroll
            for (int j = 0; j < TT; ++j)
              if (j < t.count) xch[j * 64 + row - 64] = acc[j] * ws;
          }
          if (!group_sync()) break;
          if (row < 64 && f < a.F) {
#pragma unroll
            for (int j = 0; j < TT; ++j)
              if (j < t.count)
                a.h[static_cast<int64_t>(order[t.first + j]) * a.Fp + f] =
                    activate(acc[j] * ws, a.gelu) * xch[j * 64 + row];
          }
          if (!group_sync()) break;  // before the next item's sums
        }
      } else {
        const int d = r * kRows + row;
        if (d < a.D) {
#pragma unroll
          for (int j = 0; j < TT; ++j)
            if (j < t.count)
              __stcg(a.part + (static_cast<int64_t>(sp) * pairs +
                               order[t.first + j]) * a.Dp + d,
                     acc[j] * ws);
        }
        // The parts are visible before the count that announces them.
        __threadfence();
        if (!group_sync()) break;
        unsigned *last = reinterpret_cast<unsigned *>(xch);
        if (row < t.count) {
          const int tok = order[t.first + row] / a.k;
          const unsigned before = atomicAdd(
              a.counters + static_cast<int64_t>(tok) * rb + r, 1u);
          last[row] = before + 1 == static_cast<unsigned>(tok_parts[tok] * split)
                          ? static_cast<unsigned>(tok) : 0xffffffffu;
        }
        __threadfence();
        if (!group_sync()) break;
        for (int j = 0; j < t.count; ++j) {
          const unsigned tok = last[j];
          if (tok == 0xffffffffu || d >= a.D) continue;
          float out = 0.0f;
          for (int q = 0; q < a.k; ++q) {
            const int64_t pair = static_cast<int64_t>(tok) * a.k + q;
            if (__ldcg(a.ids + pair) < 0) continue;
            float sum = 0.0f;
            for (int s2 = 0; s2 < split; ++s2)
              sum += __ldcg(a.part + (s2 * static_cast<int64_t>(pairs) + pair) *
                                         a.Dp + d);
            out = fmaf(__ldcg(a.weights + pair), sum, out);
          }
          const __nv_bfloat16 o = __float2bfloat16_rn(out);
          a.y[tok * a.ldy + d] = *reinterpret_cast<const uint16_t *>(&o);
        }
        if (!group_sync()) break;  // before the next item's list
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// Expert weights [E][rows][K] as boxes of `box_rows` rows x 128 K.
bool encode_weights(CUtensorMap *m, const uint8_t *w, int64_t K, int64_t rows,
                    int64_t E, int64_t ld, int64_t stride, uint32_t box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K),
                              static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(E)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld),
                                 static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[3] = {BK, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(w), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TT, bool UP>
fp8la_status launch_stage(const CUtensorMap &tm, const LayerArgs &a, int grid,
                          cudaStream_t s) {
  auto kern = moe_stage_kernel<TT, UP>;
  constexpr int slot = 8 + (TT == 16 ? 0 : 2) + (UP ? 0 : 1);
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<TT>::kAlloc);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  // Each kernel's set-up overlaps the one before it; the down kernel also
  // starts to read its weights (see pdl_wait above for what it waits for).
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<TT>::kAlloc;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, tm, a) != cudaSuccess) return FP8LA_ERR_CUDA;
  return FP8LA_OK;
}

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

// Most parts that K may be cut into.  Cutting pays only where there are few
// items, that is few pairs; the limit keeps the parts' memory in bounds.
int split_limit(int64_t pairs, int64_t D, int64_t F) {
  const int64_t bytes = pairs * (2 * round16(F) + round16(D)) * 4;
  const int64_t most = (int64_t(128) << 20) / (bytes > 0 ? bytes : 1);
  return most < 1 ? 1 : most > kMaxSplit ? kMaxSplit : static_cast<int>(most);
}

struct Layout {
  int64_t counters, h, part, total;
};
Layout layout(int64_t T, int64_t k, int64_t D, int64_t F) {
  const int64_t pairs = T * k;
  const int S = split_limit(pairs, D, F);
  Layout l;
  l.counters = 0;
  l.h = (T * ((D + BM - 1) / BM) * 4 + 255) / 256 * 256;
  const int64_t h = pairs * round16(F) * (S > 1 ? 2 * S : 1);
  l.part = l.h + (h * 4 + 255) / 256 * 256;
  l.total = l.part + (pairs * round16(D) * S * 4 + 255) / 256 * 256;
  return l;
}

constexpr int64_t kMaxDim = int64_t(1) << 20;

}  // namespace
}  // namespace fp8la

using namespace fp8la;

extern "C" int64_t fp8_moe_layer_workspace_bytes(int64_t tokens, int32_t top_k,
                                                 int64_t D, int64_t F) {
  if (tokens < 0 || top_k < 1 || D < 0 || F < 0) return FP8LA_ERR_INVALID_ARG;
  if (tokens > kMaxTokens || top_k > kMaxTopK || D > kMaxDim || F > kMaxDim)
    return FP8LA_ERR_UNSUPPORTED;
  return layout(tokens, top_k, D, F).total;
}

extern "C" fp8la_status fp8_moe_layer(
    const void *x, int32_t x_dtype, int64_t tokens, int64_t D, int64_t ldx,
    const int32_t *ids, const float *weights, int32_t top_k,
    int32_t num_experts, const uint8_t *w13, int64_t ld13,
    int64_t expert_stride13, const float *scale13, const uint8_t *w2,
    int64_t ld2, int64_t expert_stride2, const float *scale2, int64_t F,
    int32_t format, int32_t activation, uint16_t *y, int64_t ldy,
    void *workspace, int64_t workspace_bytes, fp8la_stream_t stream) {
  if ((x_dtype != FP8LA_TYPE_F32 && x_dtype != FP8LA_TYPE_BF16) ||
      (format != FP8LA_FORMAT_E4M3 && format != FP8LA_FORMAT_E5M2) ||
      (activation != FP8LA_ACT_SILU && activation != FP8LA_ACT_GELU_TANH))
    return FP8LA_ERR_INVALID_ARG;
  if (tokens < 0 || D < 1 || F < 1 || top_k < 1 || num_experts < 1 || ldx < D ||
      ldy < D || ld13 < D || ld2 < F)
    return FP8LA_ERR_INVALID_ARG;
  if (tokens > kMaxTokens || top_k > kMaxTopK || num_experts > kMaxExperts ||
      D > kMaxDim || F > kMaxDim || ld13 >= (int64_t(1) << 31) ||
      ld2 >= (int64_t(1) << 31) || expert_stride13 >= (int64_t(1) << 39) ||
      expert_stride2 >= (int64_t(1) << 39))
    return FP8LA_ERR_UNSUPPORTED;
  if (num_experts > 1 &&
      (expert_stride13 < 2 * F * ld13 || expert_stride2 < D * ld2))
    return FP8LA_ERR_INVALID_ARG;
  if (tokens == 0) return FP8LA_OK;
  const Layout l = layout(tokens, top_k, D, F);
  if (!x || !ids || !weights || !w13 || !scale13 || !w2 || !scale2 || !y ||
      !workspace || workspace_bytes < l.total)
    return FP8LA_ERR_INVALID_ARG;
  const int xs = x_dtype == FP8LA_TYPE_BF16 ? 2 : 4;
  if (!aligned16(w13) || !aligned16(w2) || ld13 % 16 != 0 || ld2 % 16 != 0 ||
      (num_experts > 1 && (expert_stride13 % 16 != 0 || expert_stride2 % 16 != 0)) ||
      !aligned16(workspace) || reinterpret_cast<uintptr_t>(x) % xs != 0 ||
      reinterpret_cast<uintptr_t>(y) % 2 != 0)
    return FP8LA_ERR_ALIGNMENT;
  if (!device_is_sm10x()) return FP8LA_ERR_UNSUPPORTED;
  // A single expert's stride addresses nothing, but the tensor map wants one.
  const int64_t st13 = num_experts > 1 ? expert_stride13 : 2 * F * ld13;
  const int64_t st2 = num_experts > 1 ? expert_stride2 : D * ld2;
  CUtensorMap tm13, tm2;
  if (!encode_weights(&tm13, w13, D, 2 * F, num_experts, ld13, st13, BM / 2) ||
      !encode_weights(&tm2, w2, F, D, num_experts, ld2, st2, BM))
    return FP8LA_ERR_CUDA;
  unsigned *status = status_word_ptr();
  const int grid = sm_count();
  if (!status || grid <= 0) return FP8LA_ERR_CUDA;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  LayerArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.x_bf16 = x_dtype == FP8LA_TYPE_BF16;
  a.x_vec = aligned16(x) && ldx * xs % 16 == 0;
  a.T = static_cast<int32_t>(tokens);
  a.E = num_experts;
  a.k = top_k;
  a.D = static_cast<int32_t>(D);
  a.F = static_cast<int32_t>(F);
  a.ids = ids;
  a.weights = weights;
  a.s13 = scale13;
  a.s2 = scale2;
  a.counters = reinterpret_cast<unsigned *>(ws + l.counters);
  a.h = reinterpret_cast<float *>(ws + l.h);
  a.Fp = round16(F);
  a.part = reinterpret_cast<float *>(ws + l.part);
  a.Dp = round16(D);
  a.y = y;
  a.ldy = ldy;
  a.gelu = activation == FP8LA_ACT_GELU_TANH;
  a.fmt_bits = format == FP8LA_FORMAT_E5M2 ? 1u << 7 : 0u;  // A's format
  a.max_split = split_limit(tokens * top_k, D, F);
  a.status = status;
  a.timeout_ns = wait_timeout_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  fp8la_status st;
  if (tokens <= 16) {
    st = launch_stage<16, true>(tm13, a, grid, s);
    if (st == FP8LA_OK) st = launch_stage<16, false>(tm2, a, grid, s);
  } else {
    st = launch_stage<64, true>(tm13, a, grid, s);
    if (st == FP8LA_OK) st = launch_stage<64, false>(tm2, a, grid, s);
  }
  return st == FP8LA_OK ? launch_status() : st;
}

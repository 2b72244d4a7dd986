// Mixture-of-experts layer for a few tokens, with the expert weights in FP8
// and the activations at full precision.
//
//   gate/up kernel:  [g; u] = s13[e] * W13[e] x_t,  h = act(g) * u
//   down kernel:     y_t = sum_j w_tj * s2[e_j] * (W2[e_j] h_tj)
//
// Bound: the weights of the touched experts, read once from HBM (3 D F bytes
// an expert); a few tokens do 2 flops with each byte for each token.  So both
// kernels are one stream of weight tiles from HBM through TMA into shared
// memory and straight into tcgen05.mma, with no register in between.
//
// Weights are the M side of the MMA, tokens the N side, which may be as narrow
// as 16 columns.  kind::f8f6f4 wants FP8 on both sides, so an activation
// enters as the sum of two E4M3 values,
//   v * 2^(7-e) = hi + lo / 32,   2^e <= the largest |v| < 2^(e+1),
// two columns of the MMA whose results the epilogue adds.  hi and lo keep 8
// significant bits: exact for BF16 activations down to 2^-15 of the largest
// (below that the error is under 2^-22 of the largest), and for FP32 ones no
// worse than a rounding to BF16.  A power of two as scale rounds nothing.  x
// has one scale for each token, h one for each token and 128 elements.
//
// Four launches, each with its set-up under the one before:
//   prepare  sorts the pairs by expert into tiles of up to TT and splits the
//            tokens' x into codes, one row for each pair, in that order
//   gate/up  one item = a tile x (128 gate + the same 128 up rows).  Its
//            epilogue has all 128 h of a down K block at hand, so it writes h
//            as codes with their scale.
//   down     one item = a tile x 256 rows.  The scale of h changes every 128
//            K, so its epilogue adds 128-wide partial sums in FP32 registers
//            (double-buffered in TMEM).  It starts to read weights while the
//            gate/up kernel is finishing.
//   combine  adds each token's experts, weighted, and rounds once.
// The GEMM kernels run one CTA per SM.  All items' K stages in a row are cut
// into equal ranges, one for each CTA, so every SM streams the same number of
// weight bytes whatever the sizes; a CTA's first and last item may be shared
// with its neighbours.  The parts of a shared item go to memory in FP32 and
// are added in the order of the CTAs: of h by the CTA that brings the last
// one, of y by the combine kernel.  The result does not depend on timing.
//
// Roles: warps 0-7 epilogue (TMEM lane quarter = warp % 4), warp 8 producer,
// warp 9 MMA issuer.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fp8la {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = kEpiWarps;
constexpr int kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kPrepThreads = 256;
constexpr int kPrepWarps = kPrepThreads / 32;
constexpr int BM = 128;             // weight rows of an MMA
constexpr int BK = 128;             // K of a stage (bytes = FP8 values)
constexpr int kABytes = 2 * BM * BK;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTokens = 128;
constexpr int kMaxTopK = 16;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kSlack = 64;          // positions past the last pair that are read

// TT: most tokens of a tile.
template <int TT>
struct Cfg {
  static constexpr int STAGES = TT == 16 ? 6 : 4;
  static constexpr int kBBytes = 2 * TT * BK;      // hi and lo rows
  static constexpr int kScaleBytes = 4 * TT;       // h's scales (down kernel)
  static constexpr int kTmemCols = 8 * TT;         // 2 buffers x 2 blocks x 2 TT
  static constexpr int kA = 0;
  static constexpr int kB = kA + STAGES * kABytes;
  static constexpr int kScale = kB + STAGES * kBBytes;
  static constexpr int kTop = kScale + STAGES * kScaleBytes;  // [4][TT] words
  static constexpr int kBar = kTop + 4 * TT * 4;
  static constexpr int kNumBars = 2 * STAGES + 6;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kEnd = kMisc + 32;
  static constexpr int kAlloc = kEnd + 1024;
  static_assert(kB % 1024 == 0 && kBBytes % 1024 == 0, "swizzle atoms");
  static_assert(kScale % 16 == 0 && kBar % 8 == 0, "alignment");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

struct Tile {            // up to TT pairs of one expert, at consecutive positions
  int32_t expert, first, count, pad;
};

// What the prepare kernel leaves for the others, and what passes between
// them.  Positions are places in expert order; a tile's first one is a
// multiple of 4, so that its scales are 16-byte aligned.
struct Plan {
  int32_t *n_tiles;      // [1], -1: an id is out of range, nothing is written
  Tile *tiles;
  int32_t *pos;          // [pairs], -1: no expert
  int32_t *tile_of;      // [pairs]
  unsigned *arrived;     // [tiles][row blocks]: parts of a shared h item
  uint8_t *xc;           // [2][positions][Dc] codes of x
  float *xs;             // [positions]
  uint8_t *hc;           // [2][positions][Fc] codes of h
  float *hs;             // [128-blocks of F][positions]
  float *parts;          // [CTAs][2][TT][256] parts of shared items
  float *out;            // [positions][Dc] sums of whole down items
};

struct LayerArgs {
  Plan p;
  const void *x;
  int64_t ldx;
  int32_t x_bf16, x_vec;
  int32_t T, E, k, D, F;
  int32_t P;             // positions, as allocated
  int64_t Dc, Fc;        // D and F rounded up to 16
  const int32_t *ids;
  const float *weights;
  const float *s13, *s2;
  uint16_t *y;
  int64_t ldy;
  int32_t gelu;
  uint32_t fmt_bits;
  int32_t grid;          // CTAs of the GEMM kernels
  unsigned *status;
  uint64_t timeout_ns;
};

// Ranges of the stages: stage u of `units` belongs to CTA owner(u).  Where
// there are fewer stages than CTAs, the first CTAs get one each, so that the
// CTAs that share an item always follow one another.
struct Ranges {
  int64_t units;
  int grid;
  __device__ __forceinline__ Ranges(int64_t n, int ctas)
      : units(n), grid(static_cast<int>(min(n, static_cast<int64_t>(ctas)))) {}
  __device__ __forceinline__ int64_t begin(int cta) const {
    return cta >= grid ? units : units * cta / grid;
  }
  __device__ __forceinline__ int owner(int64_t u) const {
    return static_cast<int>((grid * (u + 1) - 1) / units);
  }
};

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

// Scale of a group whose largest |v| has the bits `top` (NaN and infinity are
// the largest): v * inv lies in (-256, 256), scale = 1 / inv.  A group that
// holds an infinity or NaN is multiplied by 0, which makes those elements NaN
// and with them every output they reach.
__device__ __forceinline__ void group_scale(uint32_t top, float &inv, float &scale) {
  const uint32_t eb = max(top >> 23, 8u);
  inv = eb == 255u ? 0.0f : __uint_as_float((261u - eb) << 23);
  scale = eb == 255u ? 1.0f : __uint_as_float((eb - 7u) << 23);
}

// (a, b) scaled -> their hi codes and their lo codes (two in 16 bits each).
__device__ __forceinline__ void split_codes(float a, float b, uint32_t &hi,
                                            uint32_t &lo) {
  hi = cvt_e4m3x2(a, b);
  const float2 back = decode_e4m3x2(hi);
  lo = cvt_e4m3x2((a - back.x) * 32.0f, (b - back.y) * 32.0f);
}

// 16 TMEM columns: the hi and the lo sums of 8 tokens.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&u)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3]), "=f"(u[4]), "=f"(u[5]),
        "=f"(u[6]), "=f"(u[7]), "=f"(u[8]), "=f"(u[9]), "=f"(u[10]),
        "=f"(u[11]), "=f"(u[12]), "=f"(u[13]), "=f"(u[14]), "=f"(u[15])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ float activate(float g, int gelu) {
  if (gelu) {
    const float t = tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g));
    return 0.5f * g * (1.0f + t);
  }
  return g / (1.0f + __expf(-g));
}

// 16 elements of a token from d on, as loaded (BF16: the first 8 words), and
// their values.
__device__ __forceinline__ void load_x16(const LayerArgs &a, int t, int d,
                                         uint32_t (&w)[16]) {
  const int64_t at = static_cast<int64_t>(t) * a.ldx + d;
  if (a.x_bf16) {
    const uint16_t *p = static_cast<const uint16_t *>(a.x) + at;
    if (a.x_vec && d + 16 <= a.D) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = *(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = (d + 2 * i < a.D ? p[2 * i] : 0) |
               (d + 2 * i + 1 < a.D ? p[2 * i + 1] : 0) << 16;
    }
  } else {
    const float *p = static_cast<const float *>(a.x) + at;
    if (a.x_vec && d + 16 <= a.D) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = *(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = d + i < a.D ? __float_as_uint(p[i]) : 0;
    }
  }
}
__device__ __forceinline__ float x_value(const uint32_t (&w)[16], int bf16, int i) {
  return __uint_as_float(
      !bf16 ? w[i] : i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}

// ------------------------------------------------------------------ prepare
// Every CTA sorts the pairs by itself (places come from counts, so all CTAs
// agree); the first one writes the plan, and all of them share out the tokens.
template <int TT>
__global__ void __launch_bounds__(kPrepThreads)
    moe_prepare_kernel(const LayerArgs a) {
  __shared__ uint16_t by_warp[kPrepWarps][kMaxExperts];
  __shared__ uint16_t first_pos[kMaxExperts], first_tile[kMaxExperts];
  __shared__ int16_t pos_of[kMaxPairs];
  __shared__ int warp_sums[2][kPrepWarps];
  __shared__ uint32_t tops[kPrepWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = a.T * a.k;
  const int groups = (pairs + 31) / 32;
  const int plan_warps = min(kPrepWarps, groups);
  for (int w = 0; w < plan_warps; ++w)
    for (int e = threadIdx.x; e < a.E; e += kPrepThreads) by_warp[w][e] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  // The first token's x is on its way while the plan is made.
  constexpr int kRound = 16 * kPrepThreads;
  uint32_t xw[16];
  if (16 * threadIdx.x < a.D) load_x16(a, blockIdx.x, 16 * threadIdx.x, xw);
  bool bad = false;
  const int g_lo = warp < plan_warps ? groups * warp / plan_warps : 0;
  const int g_hi = warp < plan_warps ? groups * (warp + 1) / plan_warps : 0;
  for (int gr = g_lo; gr < g_hi; ++gr) {
    const int p = 32 * gr + lane;
    int id = p < pairs ? a.ids[p] : -1;
    if (id < -1 || id >= a.E) {
      bad = true;
      id = -1;
    }
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    if (id >= 0 && (same & ((1u << lane) - 1u)) == 0)
      by_warp[warp][id] = static_cast<uint16_t>(by_warp[warp][id] + __popc(same));
    __syncwarp();
  }
  bad = __syncthreads_or(bad);
  // Scan over the experts: pairs (low half) and tiles (high half) in one word,
  // padded positions in another.
  constexpr int kPer = kMaxExperts / kPrepThreads;
  int c[kPer], sum = 0, padded = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    c[i] = 0;
    if (e < a.E)
      for (int w = 0; w < plan_warps; ++w) c[i] += by_warp[w][e];
    sum += c[i] | ((c[i] + TT - 1) / TT) << 16;
    padded += (c[i] + 3) & ~3;
  }
  int incl = sum, pincl = padded;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    const int q = __shfl_up_sync(0xffffffffu, pincl, d);
    if (lane >= d) {
      incl += o;
      pincl += q;
    }
  }
  if (lane == 31) {
    warp_sums[0][warp] = incl;
    warp_sums[1][warp] = pincl;
  }
  __syncthreads();
  int at = incl - sum, pat = pincl - padded, all = 0;
#pragma unroll
  for (int w = 0; w < kPrepWarps; ++w) {
    const int v = warp_sums[0][w];
    if (w < warp) {
      at += v;
      pat += warp_sums[1][w];
    }
    all += v;
  }
  const int n_tiles = bad ? 0 : all >> 16;
  const bool first_cta = blockIdx.x == 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e < a.E && c[i] > 0) {
      // From here on: where each warp's next pair of the expert goes, its
      // first position and its first tile.
      int next = 0;
      for (int w = 0; w < plan_warps; ++w) {
        const int n = by_warp[w][e];
        by_warp[w][e] = static_cast<uint16_t>(next);
        next += n;
      }
      first_pos[e] = static_cast<uint16_t>(pat);
      first_tile[e] = static_cast<uint16_t>(at >> 16);
      if (first_cta && !bad) {
        int t = at >> 16;
        for (int done = 0; done < c[i]; done += TT, ++t)
          a.p.tiles[t] = {e, pat + done, min(TT, c[i] - done), 0};
      }
    }
    at += c[i] | ((c[i] + TT - 1) / TT) << 16;
    pat += (c[i] + 3) & ~3;
  }
  __syncthreads();
  for (int gr = g_lo; gr < g_hi; ++gr) {
    const int p = 32 * gr + lane;
    const int id = p < pairs && !bad ? a.ids[p] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int pos = -1, tile = 0;
    if (id >= 0) {
      const int place = by_warp[warp][id] + rank;
      pos = first_pos[id] + place;
      tile = first_tile[id] + place / TT;
    }
    if (p < pairs) {
      pos_of[p] = static_cast<int16_t>(pos);
      if (first_cta) {
        a.p.pos[p] = pos;
        a.p.tile_of[p] = tile;
      }
    }
    __syncwarp();
    if (id >= 0 && rank == 0)
      by_warp[warp][id] = static_cast<uint16_t>(by_warp[warp][id] + __popc(same));
    __syncwarp();
  }
  if (first_cta && threadIdx.x == 0) {
    *a.p.n_tiles = bad ? -1 : n_tiles;
    if (bad) atomicOr(a.status, kStatusBadDeviceArg);
  }
  const int cells = n_tiles * ((a.F + BM - 1) / BM);
  for (int i = blockIdx.x * kPrepThreads + threadIdx.x; i < cells;
       i += gridDim.x * kPrepThreads)
    a.p.arrived[i] = 0;

  // Codes of x: each token's once, written to the rows of all its pairs.
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    uint32_t top = 0;
    for (int d = 16 * threadIdx.x; d < a.D; d += kRound) {
      if (t != blockIdx.x || d >= kRound) load_x16(a, t, d, xw);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        top = max(top, __float_as_uint(x_value(xw, a.x_bf16, i)) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();  // of pos_of too, in the first round
    if (lane == 0) tops[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPrepWarps; ++w) top = max(top, tops[w]);
    float inv, scale;
    group_scale(top, inv, scale);
    if (threadIdx.x < a.k && pos_of[t * a.k + threadIdx.x] >= 0)
      a.p.xs[pos_of[t * a.k + threadIdx.x]] = scale;
    for (int d = 16 * threadIdx.x; d < a.D; d += kRound) {
      if (t != blockIdx.x || a.D > kRound) load_x16(a, t, d, xw);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h0, h1, l0, l1;
        split_codes(x_value(xw, a.x_bf16, 4 * i) * inv,
                    x_value(xw, a.x_bf16, 4 * i + 1) * inv, h0, l0);
        split_codes(x_value(xw, a.x_bf16, 4 * i + 2) * inv,
                    x_value(xw, a.x_bf16, 4 * i + 3) * inv, h1, l1);
        hi[i] = h0 | h1 << 16;
        lo[i] = l0 | l1 << 16;
      }
      for (int j = 0; j < a.k; ++j) {
        const int pos = pos_of[t * a.k + j];
        if (pos < 0) continue;
        // A row's codes past D, up to its padded end, are zeros.
        uint8_t *row = a.p.xc + static_cast<int64_t>(pos) * a.Dc + d;
        *reinterpret_cast<uint4 *>(row) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(row + static_cast<int64_t>(a.P) * a.Dc) =
            make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
}

// ------------------------------------------------------------ gate/up, down
template <int TT, bool UP>
__global__ void __launch_bounds__(kThreads, 1)
    moe_gemm_kernel(const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmC, const LayerArgs a) {
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
  auto accfull_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + b); };
  auto accfree_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 2 + b); };
  const uint32_t group_bar = bar0 + 8u * (2 * C::STAGES + 4);
  const uint32_t final_bar = bar0 + 8u * (2 * C::STAGES + 5);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sbase + C::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + C::kMisc + 4);
  volatile int *last_flag = reinterpret_cast<volatile int *>(sbase + C::kMisc + 8);
  uint32_t *tops = reinterpret_cast<uint32_t *>(sbase + C::kTop);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      // The down kernel's epilogue reads the stage's scales.
      mbar_init(empty_bar(s), UP ? 1 : 1 + kEpiWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accfull_bar(b), 1);
      mbar_init(accfree_bar(b), kEpiWarps);
    }
    mbar_init(group_bar, kEpiWarps);
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmC);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The gate/up kernel needs the plan at once.  The down kernel can only have
  // started after every CTA of the gate/up kernel passed this point, so the
  // plan is final for it too; it waits where it first needs h.
  if (UP) {
    pdl_wait();
    pdl_launch_dependents();
  }
  const int n_tiles = max(0, __ldcg(a.p.n_tiles));
  const int K = UP ? a.D : a.F;
  const int rows = UP ? a.F : a.D;          // output rows (h or y)
  constexpr int kRows = UP ? BM : 2 * BM;   // of an item
  const int nk = (K + BK - 1) / BK;
  const int rb = (rows + kRows - 1) / kRows;
  const Ranges ranges(static_cast<int64_t>(n_tiles) * rb * nk, a.grid);
  const int64_t u0 = ranges.begin(blockIdx.x), u1 = ranges.begin(blockIdx.x + 1);
  const uint32_t tmem_base = *tmem_slot;

  // The CTA's share of the item that holds stage u: the tile is innermost
  // (tiles of one expert are neighbours, so its weights are still in L2 for
  // the second), then the row block.
  struct Item {
    Tile t;
    int64_t index;
    int tile, r, c0, c1, npad;
  };
  auto item = [&](int64_t u) {
    Item w;
    w.index = u / nk;
    w.c0 = static_cast<int>(u - w.index * nk);
    w.c1 = static_cast<int>(min(static_cast<int64_t>(nk), u1 - w.index * nk));
    w.r = static_cast<int>(w.index / n_tiles);
    w.tile = static_cast<int>(w.index - static_cast<int64_t>(w.r) * n_tiles);
    const int4 v = __ldcg(reinterpret_cast<const int4 *>(a.p.tiles + w.tile));
    w.t = {v.x, v.y, v.z, v.w};
    w.npad = (w.t.count + 7) & ~7;
    return w;
  };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      auto load_w = [&](const Item &w, int c, uint32_t s) {
        const uint32_t dst = base + C::kA + s * kABytes;
        const uint32_t bytes = kABytes + 2 * w.npad * BK + (UP ? 0 : 4 * w.npad);
        mbar_arrive_expect_tx(full_bar(s), bytes);
        const int r0 = w.r * kRows;
        tma_load_3d(dst, &tmW, full_bar(s), c * BK, r0, w.t.expert);
        tma_load_3d(dst + kABytes / 2, &tmW, full_bar(s), c * BK,
                    UP ? a.F + r0 : r0 + BM, w.t.expert);
      };
      // Codes of the tile, 8 positions at a time: 8 hi rows, 8 lo rows.
      auto load_codes = [&](const Item &w, int c, uint32_t s) {
        for (int j = 0; j < w.npad; j += 8)
          tma_load_3d(base + C::kB + s * C::kBBytes + 2 * j * BK, &tmC,
                      full_bar(s), c * BK, w.t.first + j, 0);
        if (!UP)
          bulk_load(base + C::kScale + s * C::kScaleBytes,
                    a.p.hs + static_cast<int64_t>(c) * a.P + w.t.first,
                    4 * w.npad, full_bar(s));
      };
      // The down kernel fills its ring with weights before it waits for h.
      int ahead = 0;
      if (!UP) {
        for (int64_t u = u0; u < u1 && ahead < C::STAGES;) {
          const Item w = item(u);
          for (int c = w.c0; c < w.c1 && ahead < C::STAGES; ++c, ++u)
            load_w(w, c, ahead++);
        }
        pdl_wait();
        pdl_launch_dependents();
      }
      uint32_t s = 0, ph = 0, issued = 0;
      bool ok = true;
      for (int64_t u = u0; ok && u < u1;) {
        const Item w = item(u);
        u += w.c1 - w.c0;
        for (int c = w.c0; c < w.c1; ++c) {
          if (ahead > 0) {
            --ahead;
          } else {
            if (!mbar_wait(empty_bar(s), ph ^ 1u, a.timeout_ns, a.status,
                           abort_flag)) {
              ok = false;
              break;
            }
            load_w(w, c, s);
          }
          load_codes(w, c, s);
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
    // An accumulator buffer holds a whole item (gate/up) or a stage (down).
    if (lane == 0) {
      uint32_t s = 0, ph = 0, g = 0;
      bool ok = true;
      for (int64_t u = u0; ok && u < u1;) {
        const Item w = item(u);
        u += w.c1 - w.c0;
        const uint32_t idesc = idesc_e4m3_f32(BM, 2 * w.npad) | a.fmt_bits;
        for (int c = w.c0; c < w.c1; ++c) {
          const uint32_t b = g & 1u;
          if (!UP || c == w.c0)
            ok = mbar_wait(accfree_bar(b), ((g >> 1) & 1u) ^ 1u, a.timeout_ns,
                           a.status, abort_flag);
          ok = ok && mbar_wait(full_bar(s), ph, a.timeout_ns, a.status, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t adesc = smem_desc_k128_sw128(base + C::kA + s * kABytes);
          const uint64_t bdesc = smem_desc_k128_sw128(base + C::kB + s * C::kBBytes);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < BK / 32; ++q)
              umma_f8f6f4(tmem_base + (b * 2 + m) * 2 * TT,
                          adesc + m * (kABytes / 2 / 16) + 2u * q, bdesc + 2u * q,
                          idesc, (q > 0 || (UP && c > w.c0)) ? 1u : 0u);
          umma_commit(empty_bar(s));
          if (++s == C::STAGES) { s = 0; ph ^= 1u; }
          if (!UP || c + 1 == w.c1) {
            umma_commit(accfull_bar(b));
            ++g;
          }
        }
      }
      umma_commit(final_bar);
      mbar_wait_drain(final_bar, 0, a.timeout_ns, a.status);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    if (!UP) pdl_wait();
    const int quarter = warp & 3, half = warp >> 2;
    const int row = 32 * quarter + lane;  // TMEM lane
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t gph = 0;
    // Barrier of the eight warps, with a limit.
    auto group_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(group_bar);
      const bool ok = mbar_wait(group_bar, gph, a.timeout_ns, a.status, abort_flag);
      gph ^= 1u;
      return __all_sync(0xffffffffu, ok) != 0;
    };
    uint32_t g = 0, s = 0;
    bool ok = true;
    for (int64_t u = u0; ok && u < u1;) {
      const Item w = item(u);
      u += w.c1 - w.c0;
      // Where a part of a shared item goes: slot 0 if it began in an earlier
      // CTA, else 1.
      const bool shared = w.c0 > 0 || w.c1 < nk;
      float *mine = a.p.parts +
                    (static_cast<int64_t>(blockIdx.x) * 2 + (w.c0 > 0 ? 0 : 1)) *
                        TT * 256;
      if (UP) {
        // Tokens in groups of 8; the two halves of the warps take turns.  A
        // thread has one h row; gate sums are block 0, up sums block 1.
        constexpr int kG = TT / 16;
        const int f = w.r * kRows + row;
        const float ws = __ldg(a.s13 + w.t.expert);
        float gs[kG][8], us[kG][8];
#pragma unroll
        for (int q = 0; q < kG; ++q) {
          const int j0 = 16 * q + 8 * half;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            gs[q][j] = j0 < w.npad ? __ldcg(a.p.xs + w.t.first + j0 + j) : 0.0f;
        }
        const uint32_t b = g & 1u;
        const bool ready = mbar_wait(accfull_bar(b), (g >> 1) & 1u, a.timeout_ns,
                                     a.status, abort_flag);
        if (!__all_sync(0xffffffffu, ready)) break;
        ++g;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < kG; ++q) {
          const int j0 = 16 * q + 8 * half;
          if (j0 < w.npad) {
            float vg[16], vu[16];
            tmem_ld16(lane_base + b * 4 * TT + 2 * j0, vg);
            tmem_ld16(lane_base + b * 4 * TT + 2 * TT + 2 * j0, vu);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              us[q][j] = fmaf(vu[8 + j], 0.03125f, vu[j]) * gs[q][j] * ws;
              gs[q][j] = fmaf(vg[8 + j], 0.03125f, vg[j]) * gs[q][j] * ws;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(accfree_bar(b));
        if (shared) {
          // Leave the part; whoever brings the last one goes on with the sum.
          const int64_t v0 = w.index * nk;
          const int first = ranges.owner(v0), last = ranges.owner(v0 + nk - 1);
#pragma unroll
          for (int q = 0; q < kG; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int col = 16 * q + 8 * half + j;
              if (col < w.t.count) {
                __stcg(mine + col * 256 + row, gs[q][j]);
                __stcg(mine + col * 256 + 128 + row, us[q][j]);
              }
            }
          __threadfence();
          if (!group_sync()) break;
          if (threadIdx.x == 0)
            *last_flag = atomicAdd(a.p.arrived + w.index, 1u) ==
                         static_cast<unsigned>(last - first);
          __threadfence();
          if (!group_sync()) break;
          const bool go_on = *last_flag != 0;
          if (!group_sync()) break;  // read before the next item's
          if (!go_on) continue;
#pragma unroll
          for (int q = 0; q < kG; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j) gs[q][j] = us[q][j] = 0.0f;
          for (int p = first; p <= last; ++p) {
            const float *part = a.p.parts +
                                (static_cast<int64_t>(p) * 2 + (p > first ? 0 : 1)) *
                                    TT * 256 + row;
#pragma unroll
            for (int q = 0; q < kG; ++q)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int col = 16 * q + 8 * half + j;
                if (col < w.t.count) {
                  gs[q][j] += __ldcg(part + col * 256);
                  us[q][j] += __ldcg(part + col * 256 + 128);
                }
              }
          }
        }
        // h, its largest over the 128 rows, and the codes.
#pragma unroll
        for (int q = 0; q < kG; ++q)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int col = 16 * q + 8 * half + j;
            const float h = f < a.F && col < w.t.count
                                ? activate(gs[q][j], a.gelu) * us[q][j] : 0.0f;
            gs[q][j] = h;
            if (16 * q + 8 * half < w.npad) {
              const uint32_t top =
                  __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu);
              if (lane == 0) tops[quarter * TT + col] = top;
            }
          }
        if (!group_sync()) break;
#pragma unroll
        for (int q = 0; q < kG; ++q)
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const int col = 16 * q + 8 * half + j;
            if (col < w.t.count) {
              float v[2], scale[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t top = 0;
#pragma unroll
                for (int z = 0; z < 4; ++z) top = max(top, tops[z * TT + col + e]);
                float inv;
                group_scale(top, inv, scale[e]);
                v[e] = gs[q][j + e] * inv;
              }
              uint32_t hi, lo;
              split_codes(v[0], v[1], hi, lo);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (col + e < w.t.count) {
                  const int64_t at = static_cast<int64_t>(w.t.first + col + e) * a.Fc + f;
                  if (f < a.F) {
                    a.p.hc[at] = static_cast<uint8_t>(hi >> (8 * e));
                    a.p.hc[static_cast<int64_t>(a.P) * a.Fc + at] =
                        static_cast<uint8_t>(lo >> (8 * e));
                  }
                  if (row == 0)
                    a.p.hs[static_cast<int64_t>(w.r) * a.P + w.t.first + col + e] =
                        scale[e];
                }
            }
          }
        if (!group_sync()) break;  // tops are read before the next item's
      } else {
        float acc[TT];
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[j] = 0.0f;
        for (int c = w.c0; c < w.c1; ++c, ++g) {
          const uint32_t b = g & 1u;
          const bool ready = mbar_wait(accfull_bar(b), (g >> 1) & 1u, a.timeout_ns,
                                       a.status, abort_flag);
          if (!__all_sync(0xffffffffu, ready)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float *sc = reinterpret_cast<const float *>(
              sbase + C::kScale + s * C::kScaleBytes);
#pragma unroll
          for (int q = 0; q < TT / 8; ++q)
            if (8 * q < w.npad) {
              float v[16];
              tmem_ld16(lane_base + (b * 2 + half) * 2 * TT + 16 * q, v);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                acc[8 * q + j] = fmaf(fmaf(v[8 + j], 0.03125f, v[j]), sc[8 * q + j],
                                      acc[8 * q + j]);
            }
          tc_fence_before();
          // The scales were read by generic loads; their next fill is TMA's.
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(accfree_bar(b));
            mbar_arrive(empty_bar(s));
          }
          if (++s == C::STAGES) s = 0;
        }
        if (!ok) break;
        const float ws = __ldg(a.s2 + w.t.expert);
        const int d = w.r * kRows + half * BM + row;
        if (shared) {
#pragma unroll
          for (int j = 0; j < TT; ++j)
            if (j < w.t.count) __stcg(mine + j * 256 + half * BM + row, acc[j] * ws);
        } else if (d < a.D) {
#pragma unroll
          for (int j = 0; j < TT; ++j)
            if (j < w.t.count)
              __stcg(a.p.out + static_cast<int64_t>(w.t.first + j) * a.Dc + d,
                     acc[j] * ws);
        }
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

// ------------------------------------------------------------------ combine
// y of one token and one row block of the down kernel.
template <int TT>
__global__ void __launch_bounds__(2 * BM)
    moe_combine_kernel(const LayerArgs a) {
  const int t = blockIdx.x, r = blockIdx.y;
  const int d = r * 2 * BM + threadIdx.x;
  const int nk = (a.F + BK - 1) / BK, rb = (a.D + 2 * BM - 1) / (2 * BM);
  pdl_wait();
  const int n_tiles = __ldcg(a.p.n_tiles);
  if (n_tiles < 0) return;
  float out = 0.0f;
  const Ranges ranges(static_cast<int64_t>(n_tiles) * rb * nk, a.grid);
  for (int q = 0; q < a.k; ++q) {
    const int pair = t * a.k + q;
    const int pos = __ldcg(a.p.pos + pair);
    if (pos < 0) continue;
    const int tile = __ldcg(a.p.tile_of + pair);
    const float weight = __ldcg(a.weights + pair);
    const int64_t u = (static_cast<int64_t>(r) * n_tiles + tile) * nk;
    const int first = ranges.owner(u), last = ranges.owner(u + nk - 1);
    float sum = 0.0f;
    if (first == last) {
      if (d < a.D) sum = __ldcg(a.p.out + static_cast<int64_t>(pos) * a.Dc + d);
    } else {
      const int col = pos - __ldcg(&a.p.tiles[tile].first);
#pragma unroll 4
      for (int p = first; p <= last; ++p)
        sum += __ldcg(a.p.parts +
                      ((static_cast<int64_t>(p) * 2 + (p > first ? 0 : 1)) * TT +
                       col) * 256 + threadIdx.x);
    }
    out = fmaf(weight, sum, out);
  }
  if (d < a.D) {
    const __nv_bfloat16 o = __float2bfloat16_rn(out);
    a.y[static_cast<int64_t>(t) * a.ldy + d] =
        *reinterpret_cast<const uint16_t *>(&o);
  }
}

// Codes [outer][rows][K] as boxes of box_rows rows x 128 K, box_outer deep.
bool encode_codes(CUtensorMap *m, const uint8_t *w, int64_t K, int64_t rows,
                  int64_t outer, int64_t ld, int64_t stride, uint32_t box_rows,
                  uint32_t box_outer) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K),
                              static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld),
                                 static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[3] = {BK, box_rows, box_outer};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(w), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

// Positions: every expert's pairs rounded up to 4, and the rows that an
// 8-row box or the last scales may touch; a multiple of 4, as the scales' rows
// are read in 16-byte units.
int64_t positions(int64_t pairs, int64_t E) {
  return round16(pairs + 3 * (E < pairs ? E : pairs) + kSlack);
}

// Sizes of a tile of tokens: 16 leave more of shared memory to the weight ring.
int tile_tokens(int64_t T) { return T <= 16 ? 16 : 64; }

struct Layout {
  int64_t P, n_tiles, tile, pos, tile_of, arrived, xc, xs, hc, hs, parts, out,
      total;
};
Layout layout(int64_t T, int64_t k, int64_t E, int64_t D, int64_t F, int grid) {
  Layout l;
  const int64_t pairs = T * k, Dc = round16(D), Fc = round16(F);
  const int64_t tiles = (E < pairs ? E : pairs) + pairs / 16 + 1;
  l.P = positions(pairs, E);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  l.n_tiles = take(4);
  l.tile = take(tiles * 16);
  l.pos = take(pairs * 4);
  l.tile_of = take(pairs * 4);
  l.arrived = take(tiles * ((F + BM - 1) / BM) * 4);
  l.xc = take(2 * l.P * Dc);
  l.xs = take(l.P * 4);
  l.hc = take(2 * l.P * Fc);
  l.hs = take((F + BK - 1) / BK * l.P * 4);
  l.parts = take(static_cast<int64_t>(grid) * 2 * tile_tokens(T) * 256 * 4);
  l.out = take(l.P * Dc * 4);
  l.total = at;
  return l;
}

// CTAs of the GEMM kernels, for sizes on a machine without a GPU too.
int gemm_grid() {
  const int sms = sm_count();
  return sms > 0 ? sms : 152;
}

template <typename Kern, typename... Args>
bool launch_pdl(Kern kern, dim3 grid, int threads, int smem, cudaStream_t s,
                const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

template <int TT>
fp8la_status launch_layer(const CUtensorMap &tm13, const CUtensorMap &tmx,
                          const CUtensorMap &tm2, const CUtensorMap &tmh,
                          const LayerArgs &a, cudaStream_t s) {
  using C = Cfg<TT>;
  auto up = moe_gemm_kernel<TT, true>;
  auto down = moe_gemm_kernel<TT, false>;
  if (once_per_device(TT == 16 ? 8 : 9, [&] {
        const cudaError_t e = cudaFuncSetAttribute(
            up, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
        return e != cudaSuccess
                   ? e
                   : cudaFuncSetAttribute(
                         down, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         C::kAlloc);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  const dim3 combine(a.T, (a.D + 2 * BM - 1) / (2 * BM), 1);
  if (!launch_pdl(moe_prepare_kernel<TT>, a.T, kPrepThreads, 0, s, a) ||
      !launch_pdl(up, a.grid, kThreads, C::kAlloc, s, tm13, tmx, a) ||
      !launch_pdl(down, a.grid, kThreads, C::kAlloc, s, tm2, tmh, a) ||
      !launch_pdl(moe_combine_kernel<TT>, combine, 2 * BM, 0, s, a))
    return FP8LA_ERR_CUDA;
  return launch_status();
}

constexpr int64_t kMaxDim = int64_t(1) << 20;

}  // namespace
}  // namespace fp8la

using namespace fp8la;

extern "C" int64_t fp8_moe_layer_workspace_bytes(int64_t tokens, int32_t top_k,
                                                 int32_t num_experts, int64_t D,
                                                 int64_t F) {
  if (tokens < 0 || top_k < 1 || num_experts < 1 || D < 1 || F < 1)
    return FP8LA_ERR_INVALID_ARG;
  if (tokens > kMaxTokens || top_k > kMaxTopK || num_experts > kMaxExperts ||
      D > kMaxDim || F > kMaxDim)
    return FP8LA_ERR_UNSUPPORTED;
  return layout(tokens, top_k, num_experts, D, F, gemm_grid()).total;
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
  const int grid = gemm_grid();
  const Layout l = layout(tokens, top_k, num_experts, D, F, grid);
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
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const int64_t Dc = round16(D), Fc = round16(F);
  CUtensorMap tm13, tm2, tmx, tmh;
  if (!encode_codes(&tm13, w13, D, 2 * F, num_experts, ld13, st13, BM, 1) ||
      !encode_codes(&tm2, w2, F, D, num_experts, ld2, st2, BM, 1) ||
      !encode_codes(&tmx, ws + l.xc, D, l.P, 2, Dc, l.P * Dc, 8, 2) ||
      !encode_codes(&tmh, ws + l.hc, F, l.P, 2, Fc, l.P * Fc, 8, 2))
    return FP8LA_ERR_CUDA;
  unsigned *status = status_word_ptr();
  if (!status) return FP8LA_ERR_CUDA;
  LayerArgs a{};
  a.p.n_tiles = reinterpret_cast<int32_t *>(ws + l.n_tiles);
  a.p.tiles = reinterpret_cast<Tile *>(ws + l.tile);
  a.p.pos = reinterpret_cast<int32_t *>(ws + l.pos);
  a.p.tile_of = reinterpret_cast<int32_t *>(ws + l.tile_of);
  a.p.arrived = reinterpret_cast<unsigned *>(ws + l.arrived);
  a.p.xc = ws + l.xc;
  a.p.xs = reinterpret_cast<float *>(ws + l.xs);
  a.p.hc = ws + l.hc;
  a.p.hs = reinterpret_cast<float *>(ws + l.hs);
  a.p.parts = reinterpret_cast<float *>(ws + l.parts);
  a.p.out = reinterpret_cast<float *>(ws + l.out);
  a.x = x;
  a.ldx = ldx;
  a.x_bf16 = x_dtype == FP8LA_TYPE_BF16;
  a.x_vec = aligned16(x) && ldx * xs % 16 == 0;
  a.T = static_cast<int32_t>(tokens);
  a.E = num_experts;
  a.k = top_k;
  a.D = static_cast<int32_t>(D);
  a.F = static_cast<int32_t>(F);
  a.P = static_cast<int32_t>(l.P);
  a.Dc = Dc;
  a.Fc = Fc;
  a.ids = ids;
  a.weights = weights;
  a.s13 = scale13;
  a.s2 = scale2;
  a.y = y;
  a.ldy = ldy;
  a.gelu = activation == FP8LA_ACT_GELU_TANH;
  a.fmt_bits = format == FP8LA_FORMAT_E5M2 ? 1u << 7 : 0u;  // A's format
  a.grid = grid;
  a.status = status;
  a.timeout_ns = wait_timeout_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return tile_tokens(tokens) == 16 ? launch_layer<16>(tm13, tmx, tm2, tmh, a, s)
                                   : launch_layer<64>(tm13, tmx, tm2, tmh, a, s);
}

// Mixture-of-experts layer for a few tokens, with the expert weights in FP8
// and the activations at 8 (BF16 x) and 18 bits (FP32 x, and h).
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
// enters as a sum of E4M3 values under a power of two, which rounds nothing:
//   BF16 x     v * 2^(7-e) = t0 + t1 / 32
//   FP32 x, h  v * 2^(7-e) = t0 + t1 + (t2 + t3) / 1024
// with 2^e <= the largest |v| < 2^(e+1) of the token (x), or of the token's 128
// neighbours (h).  Each term keeps what the ones before left to 2^-5, the first
// v to 2^-4.  So two terms hold BF16's 8 bits (exact down to 2^-15 of the
// largest, off by at most 2^-22 of the largest below), and four hold 2^-19 of
// v, or 2^-27 of the largest where that is more: with two, h alone would put
// one output in five beside its BF16 neighbour.  Terms of the same scale are
// added into the same columns of the MMA, so four terms take no more of TMEM
// than two; the epilogue adds the two scales' sums.
//
// Four launches, each with its set-up under the one before:
//   prepare  sorts the pairs by expert into tiles of up to TT and splits the
//            tokens' x into codes, a row of each term for each pair, in that
//            order
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
//
// Measured on the stream, the four launches with the router's, 2 of 8 experts of
// 4096 x 14336: 80 us for 1 token (352 MB, 4.4 TB/s), 270 us for 128 tokens (1.41
// GB, 5.2 TB/s); 8 of 64 of 2048 x 1408, 24 tokens of FP32: 115 us (4.6 TB/s).
// Time stamps in the kernels, 1 / 24 / 128 tokens: first codes at 14 / 12 / 12 us,
// gate/up's MMAs until 46 / 67 / 153 in the mean CTA (its weights at 7.5, 6.5, 6.7
// TB/s), down's from 54 / 75 / 167 to 72 / 103 / 252 (6.6, 6.5, 5.5 TB/s), end of
// combine at 77 / 109 / 258.  What is left over the weights' time is the start
// (cold code and ids) and the gap in which the last parts of h are joined.  Four
// terms instead of two cost 77 -> 80, 109 -> 115 and 254 -> 270 us: fewer stages of
// weights fit beside the codes.
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
constexpr int kSlack = 64;          // positions past the last pair that are read

// Starts: three 16-bit words for each expert, and warp sums.
constexpr int kStartsBytes = kMaxExperts * 6 + 256;

// Terms of an activation, and the factor of those with the smaller scale.
constexpr int kBf16Terms = 2, kTerms = 4;
template <int TERMS>
constexpr float kSmall = TERMS == 2 ? 1.0f / 32 : 1.0f / 1024;

// TT: most tokens of a tile.
template <int TT, int TERMS>
struct Cfg {
  // As many as fit: 32 KB of weights each, beside the codes.
  static constexpr int STAGES = TERMS == 2 ? (TT == 16 ? 6 : 4) : (TT == 16 ? 5 : 3);
  static constexpr int kPairBytes = 2 * TT * BK;   // rows of a term of each scale
  static constexpr int kBBytes = TERMS / 2 * kPairBytes;
  static constexpr int kScaleBytes = 4 * TT;       // h's scales (down kernel)
  static constexpr int kTmemCols = 8 * TT;         // 2 buffers x 2 blocks x 2 TT
  static constexpr int kA = 0;
  static constexpr int kB = kA + STAGES * kABytes;
  static constexpr int kScale = kB + STAGES * kBBytes;
  static constexpr int kTop = kScale + STAGES * kScaleBytes;  // [4][TT] words
  static constexpr int kStarts = kTop + 4 * TT * 4;      // gate/up: Starts
  static constexpr int kBar = kStarts + kStartsBytes;
  static constexpr int kNumBars = 2 * STAGES + 6;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kEnd = kMisc + 32;
  static constexpr int kAlloc = kEnd + 1024;
  static_assert(kB % 1024 == 0 && kPairBytes % 1024 == 0, "swizzle atoms");
  static_assert(kMaxExperts * 4 <= STAGES * kBBytes, "the starts' counters");
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
  uint8_t *xc;           // [terms][positions][Dc] codes of x, see split_codes
  float *xs;             // [positions]
  uint8_t *hc;           // [terms][positions][Fc] codes of h
  float *hs;             // [128-blocks of F][positions]
  float *parts;          // [CTAs][2][TT][256] parts of shared items
  float *out;            // [positions][Dc] sums of whole down items
};

struct LayerArgs {
  Plan p;
  const void *x;
  int64_t ldx;
  int32_t x_vec;
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

// (a, b) scaled -> the codes of their terms (two in 16 bits each), in the order
// of the planes in memory: t0, t1, or t0, t2, t1, t3, so that each two planes
// hold a term of either scale.
template <int TERMS>
__device__ __forceinline__ void split_codes(float a, float b, uint32_t (&c)[TERMS]) {
  auto take = [&](uint32_t &code) {
    code = cvt_e4m3x2(a, b);
    const float2 back = decode_e4m3x2(code);
    a -= back.x;
    b -= back.y;
  };
  auto grow = [&]() {
    a *= 1.0f / kSmall<TERMS>;
    b *= 1.0f / kSmall<TERMS>;
  };
  take(c[0]);
  if (TERMS > 2) take(c[TERMS - 2]);
  grow();
  take(c[1]);
  if (TERMS > 2) take(c[TERMS - 1]);
}

// 16 TMEM columns: 8 tokens' sums of the terms of either scale.
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
  return __fdividef(g, 1.0f + __expf(-g));
}

// 16 elements of a token from d on, as loaded (BF16: the first 8 words), and
// their values.
template <bool F32>
__device__ __forceinline__ void load_x16(const LayerArgs &a, int t, int d,
                                         uint32_t (&w)[16]) {
  const int64_t at = static_cast<int64_t>(t) * a.ldx + d;
  if (a.x_vec && d + 16 <= a.D) {
    const uint4 *p = reinterpret_cast<const uint4 *>(
        static_cast<const char *>(a.x) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) {
      const uint4 v = p[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else if (F32) {
    const uint32_t *p = static_cast<const uint32_t *>(a.x) + at;
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = d + i < a.D ? p[i] : 0;
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(a.x) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = (d + 2 * i < a.D ? p[2 * i] : 0) |
             (d + 2 * i + 1 < a.D ? p[2 * i + 1] : 0) << 16;
  }
}
template <bool F32>
__device__ __forceinline__ float x_value(const uint32_t (&w)[16], int i) {
  return __uint_as_float(F32     ? w[i]
                         : i & 1 ? w[i >> 1] & 0xffff0000u
                                 : w[i >> 1] << 16);
}

// Where each expert's pairs and tiles begin, by a whole CTA.
struct Starts {
  uint16_t count[kMaxExperts], first_pos[kMaxExperts], first_tile[kMaxExperts];
  int warp_sums[2][32];
};

// Counts the pairs of each expert and fills *s; returns the number of tiles,
// -1 if an id is out of range.  counter: kMaxExperts words of shared memory,
// free for TMA to write afterwards.  Ends with a barrier.
template <int TT, int THREADS>
__device__ __forceinline__ int find_starts(const LayerArgs &a, Starts *s,
                                           uint32_t *counter) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.E; e += THREADS) counter[e] = 0;
  __syncthreads();
  bool bad = false;
  const int pairs = a.T * a.k;
  for (int p = threadIdx.x; p < pairs; p += THREADS) {
    const int id = __ldcg(a.ids + p);
    if (id >= 0 && id < a.E) atomicAdd(&counter[id], 1u);
    else bad |= id != -1;
  }
  if (__syncthreads_or(bad)) return -1;
  // A thread has `per` consecutive experts.  Pairs (low half) and tiles (high
  // half) are scanned in one word, padded positions in another.
  const int per = (a.E + THREADS - 1) / THREADS;
  const int e0 = threadIdx.x * per, e1 = min(e0 + per, a.E);
  int tiles = 0, padded = 0;
  for (int e = e0; e < e1; ++e) {
    const int n = static_cast<int>(counter[e]);
    tiles += (n + TT - 1) / TT;
    padded += (n + 3) & ~3;
  }
  int t_incl = tiles, p_incl = padded;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, t_incl, d);
    const int q = __shfl_up_sync(0xffffffffu, p_incl, d);
    if (lane >= d) {
      t_incl += t;
      p_incl += q;
    }
  }
  if (lane == 31) {
    s->warp_sums[0][warp] = t_incl;
    s->warp_sums[1][warp] = p_incl;
  }
  __syncthreads();
  int t_at = t_incl - tiles, p_at = p_incl - padded, all = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    const int v = s->warp_sums[0][w];
    if (w < warp) {
      t_at += v;
      p_at += s->warp_sums[1][w];
    }
    all += v;
  }
  for (int e = e0; e < e1; ++e) {
    const int n = static_cast<int>(counter[e]);
    s->count[e] = static_cast<uint16_t>(n);
    s->first_pos[e] = static_cast<uint16_t>(p_at);
    s->first_tile[e] = static_cast<uint16_t>(t_at);
    t_at += (n + TT - 1) / TT;
    p_at += (n + 3) & ~3;
  }
  fence_proxy_async_smem();
  __syncthreads();
  return all;
}

static_assert(sizeof(Starts) == kStartsBytes, "shared memory");

template <int TT>
__device__ __forceinline__ Tile tile_of_expert(const Starts *s, int e, int tile) {
  const int done = (tile - s->first_tile[e]) * TT;
  return {e, s->first_pos[e] + done, min(TT, s->count[e] - done), 0};
}

// ------------------------------------------------------------------ prepare
// One CTA for each token.  It finds the starts by itself (counts do not depend
// on order) and the places of its own pairs: the rank of a pair in its expert
// is the number of earlier pairs with the same id.
template <int TT, bool F32>
__global__ void __launch_bounds__(kPrepThreads)
    moe_prepare_kernel(const LayerArgs a) {
  __shared__ Starts s;
  __shared__ uint32_t counter[kMaxExperts];
  __shared__ int pos_of[kMaxTopK];
  __shared__ uint32_t tops[kPrepWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kRound = 16 * kPrepThreads;
  uint32_t xw[16], top = 0;
  for (int d = 16 * threadIdx.x; d < a.D; d += kRound) {
    load_x16<F32>(a, t, d, xw);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      top = max(top, __float_as_uint(x_value<F32>(xw, i)) & 0x7fffffffu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) tops[warp] = top;
  const int n_tiles = find_starts<TT, kPrepThreads>(a, &s, counter);
  if (t == 0 && threadIdx.x == 0) {
    *a.p.n_tiles = n_tiles;
    if (n_tiles < 0) atomicOr(a.status, kStatusBadDeviceArg);
  }
  if (n_tiles < 0) return;
  if (t == 0)
    for (int e = threadIdx.x; e < a.E; e += kPrepThreads)
      for (int i = s.first_tile[e], n = (s.count[e] + TT - 1) / TT; n > 0; --n, ++i)
        a.p.tiles[i] = tile_of_expert<TT>(&s, e, i);
  const int cells = n_tiles * ((a.F + BM - 1) / BM);
  for (int i = t * kPrepThreads + threadIdx.x; i < cells; i += gridDim.x * kPrepThreads)
    a.p.arrived[i] = 0;

#pragma unroll
  for (int w = 0; w < kPrepWarps; ++w) top = max(top, tops[w]);
  float inv, scale;
  group_scale(top, inv, scale);
  for (int j = warp; j < a.k; j += kPrepWarps) {
    const int pair = t * a.k + j;
    const int id = __ldcg(a.ids + pair);
    int rank = 0;
    for (int p = lane; p < pair; p += 32) rank += __ldcg(a.ids + p) == id;
    rank = __reduce_add_sync(0xffffffffu, rank);
    if (lane == 0) {
      const int pos = id < 0 ? -1 : s.first_pos[id] + rank;
      pos_of[j] = pos;
      a.p.pos[pair] = pos;
      if (id >= 0) {
        a.p.tile_of[pair] = s.first_tile[id] + rank / TT;
        a.p.xs[pos] = scale;
      }
    }
  }
  __syncthreads();
  // The token's codes, to the rows of all its pairs.  What lies between D and
  // a row's padded end becomes zeros.
  for (int d = 16 * threadIdx.x; d < a.D; d += kRound) {
    if (a.D > kRound) load_x16<F32>(a, t, d, xw);
    constexpr int kT = F32 ? kTerms : kBf16Terms;
    uint32_t w[kT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c0[kT], c1[kT];
      split_codes<kT>(x_value<F32>(xw, 4 * i) * inv, x_value<F32>(xw, 4 * i + 1) * inv,
                      c0);
      split_codes<kT>(x_value<F32>(xw, 4 * i + 2) * inv,
                      x_value<F32>(xw, 4 * i + 3) * inv, c1);
#pragma unroll
      for (int p = 0; p < kT; ++p) w[p][i] = c0[p] | c1[p] << 16;
    }
    for (int j = 0; j < a.k; ++j) {
      if (pos_of[j] < 0) continue;
#pragma unroll
      for (int p = 0; p < kT; ++p)
        *reinterpret_cast<uint4 *>(
            a.p.xc + (static_cast<int64_t>(p) * a.P + pos_of[j]) * a.Dc + d) =
            make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    }
  }
}

// ------------------------------------------------------------ gate/up, down
template <int TT, int TERMS, bool UP>
__global__ void __launch_bounds__(kThreads, 1)
    moe_gemm_kernel(const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmC, const LayerArgs a) {
  using C = Cfg<TT, TERMS>;
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
  // Neither kernel waits here for the one before it.  That one lets its
  // dependents start only after its own wait, so what precedes it is final:
  // the ids for the gate/up kernel, which finds the starts of the experts by
  // itself, and the plan for the down kernel.  So both fill their rings with
  // weights at once, and wait where they need codes.
  Starts *starts = reinterpret_cast<Starts *>(sbase + C::kStarts);
  const int n_tiles =
      max(0, UP ? find_starts<TT, kThreads>(
                      a, starts, reinterpret_cast<uint32_t *>(sbase + C::kB))
                : __ldcg(a.p.n_tiles));
  const int K = UP ? a.D : a.F;
  const int rows = UP ? a.F : a.D;          // output rows (h or y)
  constexpr int kRows = UP ? BM : 2 * BM;   // of an item
  const int nk = (K + BK - 1) / BK;
  const int rb = (rows + kRows - 1) / kRows;
  const Ranges ranges(static_cast<int64_t>(n_tiles) * rb * nk, a.grid);
  const int64_t u0 = ranges.begin(blockIdx.x), u1 = ranges.begin(blockIdx.x + 1);
  const uint32_t tmem_base = *tmem_slot;

  // The CTA's n-th item: first those that it shares with its neighbours (so
  // that their parts are long there when the kernel ends), then the others.
  // In an item's index the tile is innermost (tiles of one expert are
  // neighbours, so its weights are still in L2 for the second), then the row
  // block.
  struct Item {
    Tile t;
    int64_t index;
    int tile, r, c0, c1, npad;
  };
  const int64_t i0 = nk > 0 && u1 > u0 ? u0 / nk : 0;
  const int items = u1 > u0 ? static_cast<int>((u1 - 1) / nk - i0) + 1 : 0;
  const int head = items > 1 && u0 > i0 * nk;
  const int ends = head + (items > 1 && u1 < (i0 + items) * nk);
  auto item = [&](int n) {
    Item w;
    w.index = i0 + (n >= ends ? n - ends + head : n < head ? 0 : items - 1);
    const int64_t v = w.index * nk;
    w.c0 = static_cast<int>(max(u0 - v, static_cast<int64_t>(0)));
    w.c1 = static_cast<int>(min(u1 - v, static_cast<int64_t>(nk)));
    w.r = static_cast<int>(w.index / n_tiles);
    w.tile = static_cast<int>(w.index - static_cast<int64_t>(w.r) * n_tiles);
    if (UP) {
      // The last expert whose first tile is not after this one and that has
      // any (one without shares its first tile with the next).
      int lo = 0, hi = a.E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts->first_tile[mid] <= w.tile) lo = mid;
        else hi = mid - 1;
      }
      while (starts->count[lo] == 0) --lo;
      w.t = tile_of_expert<TT>(starts, lo, w.tile);
    } else {
      const int4 q = __ldcg(reinterpret_cast<const int4 *>(a.p.tiles + w.tile));
      w.t = {q.x, q.y, q.z, q.w};
    }
    w.npad = (w.t.count + 7) & ~7;
    return w;
  };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      auto load_w = [&](const Item &w, int c, uint32_t s) {
        const uint32_t dst = base + C::kA + s * kABytes;
        const uint32_t bytes = kABytes + TERMS * w.npad * BK + (UP ? 0 : 4 * w.npad);
        mbar_arrive_expect_tx(full_bar(s), bytes);
        const int r0 = w.r * kRows;
        tma_load_3d(dst, &tmW, full_bar(s), c * BK, r0, w.t.expert);
        tma_load_3d(dst + kABytes / 2, &tmW, full_bar(s), c * BK,
                    UP ? a.F + r0 : r0 + BM, w.t.expert);
      };
      // Codes of the tile, 8 positions and two planes at a time: 8 rows of the
      // one, 8 of the other.
      auto load_codes = [&](const Item &w, int c, uint32_t s) {
#pragma unroll
        for (int p = 0; p < TERMS; p += 2)
          for (int j = 0; j < w.npad; j += 8)
            tma_load_3d(base + C::kB + s * C::kBBytes + p / 2 * C::kPairBytes + 2 * j * BK,
                        &tmC, full_bar(s), c * BK, w.t.first + j, p);
        if (!UP)
          bulk_load(base + C::kScale + s * C::kScaleBytes,
                    a.p.hs + static_cast<int64_t>(c) * a.P + w.t.first,
                    4 * w.npad, full_bar(s));
      };
      int ahead = 0;
      for (int n = 0; n < items && ahead < C::STAGES; ++n) {
        const Item w = item(n);
        for (int c = w.c0; c < w.c1 && ahead < C::STAGES; ++c)
          load_w(w, c, ahead++);
      }
      pdl_wait();
      pdl_launch_dependents();
      uint32_t s = 0, ph = 0, issued = 0;
      bool ok = true;
      for (int n = 0; ok && n < items; ++n) {
        const Item w = item(n);
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
      for (int n = 0; ok && n < items; ++n) {
        const Item w = item(n);
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
#pragma unroll
              for (int p = 0; p < TERMS / 2; ++p)
                umma_f8f6f4(tmem_base + (b * 2 + m) * 2 * TT,
                            adesc + m * (kABytes / 2 / 16) + 2u * q,
                            bdesc + p * (C::kPairBytes / 16) + 2u * q, idesc,
                            (p > 0 || q > 0 || (UP && c > w.c0)) ? 1u : 0u);
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
    pdl_wait();
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
    uint32_t g = 0, s = 0, ph = 0;
    bool ok = true;
    for (int n = 0; ok && n < items; ++n) {
      const Item w = item(n);
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
              us[q][j] = fmaf(vu[8 + j], kSmall<TERMS>, vu[j]) * gs[q][j] * ws;
              gs[q][j] = fmaf(vg[8 + j], kSmall<TERMS>, vg[j]) * gs[q][j] * ws;
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
          if (16 * q + 8 * half < w.npad) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int col = 16 * q + 8 * half + j;
              const float h = f < a.F && col < w.t.count
                                  ? activate(gs[q][j], a.gelu) * us[q][j] : 0.0f;
              gs[q][j] = h;
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
              uint32_t code[kTerms];
              split_codes<kTerms>(v[0], v[1], code);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (col + e < w.t.count) {
                  if (f < a.F)
#pragma unroll
                    for (int p = 0; p < kTerms; ++p)
                      a.p.hc[(static_cast<int64_t>(p) * a.P + w.t.first + col + e) * a.Fc +
                             f] = static_cast<uint8_t>(code[p] >> (8 * e));
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
          // The accumulators were signalled by the MMA; the scales, which these
          // threads read themselves, by their copy.
          const bool ready = mbar_wait(full_bar(s), ph, a.timeout_ns, a.status,
                                       abort_flag) &&
                             mbar_wait(accfull_bar(b), (g >> 1) & 1u, a.timeout_ns,
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
                acc[8 * q + j] = fmaf(fmaf(v[8 + j], kSmall<TERMS>, v[j]),
                                      sc[8 * q + j], acc[8 * q + j]);
            }
          tc_fence_before();
          // The scales were read by generic loads; their next fill is TMA's.
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(accfree_bar(b));
            mbar_arrive(empty_bar(s));
          }
          if (++s == C::STAGES) { s = 0; ph ^= 1u; }
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
// y of one token and one row block of the down kernel.  The places of the
// parts follow from the plan, so they are worked out, a slot for each thread,
// before the down kernel has finished; after that one round of loads remains.
template <int TT>
__global__ void __launch_bounds__(2 * BM)
    moe_combine_kernel(const LayerArgs a) {
  __shared__ const float *part[kMaxTopK];
  __shared__ int parts[kMaxTopK];
  __shared__ float weight[kMaxTopK];
  const int t = blockIdx.x, r = blockIdx.y;
  const int d = r * 2 * BM + threadIdx.x;
  const int n_tiles = __ldcg(a.p.n_tiles);
  if (threadIdx.x < a.k) {
    const int q = threadIdx.x, pair = t * a.k + q;
    const int pos = n_tiles > 0 ? __ldcg(a.p.pos + pair) : -1;
    parts[q] = 0;
    if (pos >= 0) {
      const int nk = (a.F + BK - 1) / BK, rb = (a.D + 2 * BM - 1) / (2 * BM);
      const Ranges ranges(static_cast<int64_t>(n_tiles) * rb * nk, a.grid);
      const int tile = __ldcg(a.p.tile_of + pair);
      weight[q] = __ldcg(a.weights + pair);
      const int64_t u = (static_cast<int64_t>(r) * n_tiles + tile) * nk;
      const int first = ranges.owner(u), last = ranges.owner(u + nk - 1);
      parts[q] = last - first + 1;
      // The first CTA's part is in its slot 1, the others' in their slots 0.
      part[q] = first == last
                    ? a.p.out + static_cast<int64_t>(pos) * a.Dc + r * 2 * BM
                    : a.p.parts + ((static_cast<int64_t>(first) * 2 + 1) * TT +
                                   pos - __ldcg(&a.p.tiles[tile].first)) * 256;
    }
  }
  __syncthreads();
  pdl_wait();
  if (n_tiles < 0 || d >= a.D) return;
  float out = 0.0f;
#pragma unroll 4
  for (int q = 0; q < a.k; ++q) {
    const int n = parts[q];
    if (n == 0) continue;
    float sum = __ldcg(part[q] + threadIdx.x);
    const float *p = part[q] + TT * 256;
#pragma unroll 4
    for (int i = 1; i < n; ++i, p += 2 * TT * 256) sum += __ldcg(p + threadIdx.x);
    out = fmaf(weight[q], sum, out);
  }
  const __nv_bfloat16 o = __float2bfloat16_rn(out);
  a.y[static_cast<int64_t>(t) * a.ldy + d] = *reinterpret_cast<const uint16_t *>(&o);
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

// Tokens of a tile.  Tiles of 16 leave more of shared memory to the weight ring
// (5 or 6 stages against 3 or 4) but read the weights of an expert with more
// tokens again, from L2.  Measured, us for a layer with tiles of 16 / of 64, by the
// mean number of tokens of an expert, BF16 x, then FP32: 3 (24 tokens, 8 of 64
// experts) 113 / 122, 116 / 126; 8 (64 tokens) 121 / 131, 124 / 134; 8 (32 tokens, 2
// of 8) 137 / 139, 139 / 146; 16 (64 tokens, 2 of 8) 188 / 143, 194 / 152; 16 (128
// tokens, 8 of 64) 154 / 145, 167 / 144.
int tile_tokens(int64_t T, int64_t k, int64_t E) {
  return T <= 16 || T * k <= 8 * E ? 16 : 64;
}

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
  l.xc = take(kTerms * l.P * Dc);
  l.xs = take(l.P * 4);
  l.hc = take(kTerms * l.P * Fc);
  l.hs = take((F + BK - 1) / BK * l.P * 4);
  l.parts = take(static_cast<int64_t>(grid) * 2 * tile_tokens(T, k, E) * 256 * 4);
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

template <int TT, int XTERMS>
fp8la_status launch_layer(const CUtensorMap &tm13, const CUtensorMap &tmx,
                          const CUtensorMap &tm2, const CUtensorMap &tmh,
                          const LayerArgs &a, int slot, cudaStream_t s) {
  using CU = Cfg<TT, XTERMS>;
  using CD = Cfg<TT, kTerms>;
  auto up = moe_gemm_kernel<TT, XTERMS, true>;
  auto down = moe_gemm_kernel<TT, kTerms, false>;
  if (once_per_device(slot, [&] {
        const cudaError_t e = cudaFuncSetAttribute(
            up, cudaFuncAttributeMaxDynamicSharedMemorySize, CU::kAlloc);
        return e != cudaSuccess
                   ? e
                   : cudaFuncSetAttribute(
                         down, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         CD::kAlloc);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  const dim3 combine(a.T, (a.D + 2 * BM - 1) / (2 * BM), 1);
  if (!launch_pdl(moe_prepare_kernel<TT, XTERMS == kTerms>, a.T, kPrepThreads, 0, s,
                  a) ||
      !launch_pdl(up, a.grid, kThreads, CU::kAlloc, s, tm13, tmx, a) ||
      !launch_pdl(down, a.grid, kThreads, CD::kAlloc, s, tm2, tmh, a) ||
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
      !aligned16(workspace) || !aligned_to(x, xs) || !aligned_to(y, 2) ||
      !aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(scale13, 4) ||
      !aligned_to(scale2, 4))
    return FP8LA_ERR_ALIGNMENT;
  if (!device_is_sm10x()) return FP8LA_ERR_UNSUPPORTED;
  // A single expert's stride addresses nothing, but the tensor map wants one.
  const int64_t st13 = num_experts > 1 ? expert_stride13 : 2 * F * ld13;
  const int64_t st2 = num_experts > 1 ? expert_stride2 : D * ld2;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const int64_t Dc = round16(D), Fc = round16(F);
  const bool bf16 = x_dtype == FP8LA_TYPE_BF16;
  CUtensorMap tm13, tm2, tmx, tmh;
  if (!encode_codes(&tm13, w13, D, 2 * F, num_experts, ld13, st13, BM, 1) ||
      !encode_codes(&tm2, w2, F, D, num_experts, ld2, st2, BM, 1) ||
      !encode_codes(&tmx, ws + l.xc, D, l.P, bf16 ? kBf16Terms : kTerms, Dc, l.P * Dc, 8, 2) ||
      !encode_codes(&tmh, ws + l.hc, F, l.P, kTerms, Fc, l.P * Fc, 8, 2))
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
  if (tile_tokens(tokens, top_k, num_experts) == 16)
    return bf16 ? launch_layer<16, kBf16Terms>(tm13, tmx, tm2, tmh, a, 8, s)
                : launch_layer<16, kTerms>(tm13, tmx, tm2, tmh, a, 10, s);
  return bf16 ? launch_layer<64, kBf16Terms>(tm13, tmx, tm2, tmh, a, 9, s)
              : launch_layer<64, kTerms>(tm13, tmx, tm2, tmh, a, 11, s);
}

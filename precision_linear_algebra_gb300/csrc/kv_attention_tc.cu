// Attention of many rows over the FP8 key/value cache, on the 5th-generation tensor
// cores.  Formulas and precision as in kv_attention.cu.
//
// Bound: the tensor cores at the half rate (q and the weights are not quantised to
// FP8), and beside them the exponentials and the conversions.  A CTA takes 256 rows,
// two tiles of 128, against tiles of 128 tokens, so that one tile's products run
// while the other's weights are made:
//
//   warps 0-3, 4-7   a tile of rows each, one row a thread: scores from tensor
//                    memory, running maximum, weights as halves back over them
//   warps 8-11       K's and V's codes from the cache (any pages, 16 bytes a load) to
//                    halves in shared memory, swizzled as the MMA reads them: K with
//                    D along its rows, V the same, read as the transposed operand
//   warp 12          issues the MMAs: S = Q K^T from shared memory, O += P V with P in
//                    tensor memory
//   warps 13-15      the next rows of q, scaled by a power of two to halves (an FP32
//                    row as two terms), in place over what cp.async brought
//
// Tensor memory: S (and P over it) and O of both tiles, 512 columns with D = 128.
// O stays there; a row's is rescaled only where its maximum grew by 2^8.
//
// V codes that are not finite and that some row of the CTA does not see would reach
// it as 0 x NaN: such a tile's are written as zeros, and the rows that do see them get
// them at the end, from the cache.
#include "kv_attention.cuh"

namespace fp8la {
namespace kv {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 128;          // of a tile
constexpr int kItemRows = 256;
constexpr int kTokens = 128;        // of a tile
constexpr int kScaleBufs = 4;       // K's scales, log2 and reciprocal of V's, an exponent
constexpr int kScaleBytes = 3 * kTokens * 4 + 16;
constexpr float kShift = 7.0f;      // as in kv_attention.cu
constexpr float kLazy = 8.0f;
constexpr int kQWarps = 3;

template <int DP, int TERMS>
struct Cfg {
  static constexpr int kBlock = kRows * 128;            // 64 elements of each row
  static constexpr int kTileBytes = DP / 64 * kBlock;   // halves of a tile
  static constexpr int kQ = 2 * TERMS * kTileBytes;
  static constexpr int SLOTS = TERMS == 1 ? 3 : 2;      // K's and V's tiles in turn
  static constexpr int kRing = kQ;
  // Codes under way, in units of half a tile: K, K, V, V of the next tile, or two.
  static constexpr int UNITS = TERMS == 1 ? 4 : 2;
  static constexpr int kUnit = kTokens / 2 * DP;
  static constexpr int kRaw = kRing + SLOTS * kTileBytes;
  static constexpr int kScales = kRaw + UNITS * kUnit;
  static constexpr int kFactors = kScales + kScaleBufs * kScaleBytes;
  static constexpr int kBar = kFactors + 2 * kItemRows * 4;
  static constexpr int kBars = 2 * SLOTS + 2 * kScaleBufs + 19;
  static constexpr int kMisc = kBar + kBars * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static constexpr int kS = 0, kO = 256;                // tensor memory columns
  static_assert(kAlloc <= 224 * 1024, "shared memory");
  static_assert(kO + 2 * DP <= 512, "tensor memory");
};

// D[tmem] (+)= A B^T, halves, FP32 sums; A from shared memory, or from tensor memory.
// Executed by a whole warp, which does not branch around it: one lane issues it.
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::
          "r"(bar)
      : "memory");
}

// kind::f16 with half operands and an FP32 accumulator, M = 128; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}

// An MN-major operand: a 128-byte swizzled row of 64 elements for each K, blocks of 64
// elements `block` bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t block) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(block >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// 32 columns of this thread's lane, without a wait.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
        "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]),
        "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]),
        "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]),
        "=f"(r[30]), "=f"(r[31])
      : "r"(addr)
      : "memory");
}
// Waits for loads; the registers pass through, so that no use comes before it.
__device__ __forceinline__ void tmem_wait32(float *r) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]),
        "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]),
        "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]),
        "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
        "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27])
      :
      : "memory");
  asm volatile("" : "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const float *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31};"
      ::"f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]),
        "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]),
        "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]), "f"(r[19]),
        "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]),
        "f"(r[26]), "f"(r[27]), "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31]),
        "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Pairs of FP32 values.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Two pairs of shared memory.
__device__ __forceinline__ void lds_pairs(uint32_t a, uint64_t &x, uint64_t &y) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(a));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ int exponent_of(float v) {
  const int e = static_cast<int>(__float_as_uint(v) >> 23);
  if (v == 0.0f || e >= 255) return 0;
  return e > 0 ? e - 127 : -126;
}
__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Columns k .. k+31 of V that hold a code that is not finite at a token that a row sees,
// of the tiles that were written without such codes: those that not all rows see.
template <typename Fm>
__device__ __noinline__ uint32_t lost_columns(const AttnArgs &a, const Item &it, int seen, int k) {
  const int all = tokens_seen(a, it.q, it.rt * kItemRows);
  const int end = min(seen, (it.tile0 + it.count) * kTokens);
  uint32_t bad = 0;
  for (int j = max(it.tile0, all / kTokens) * kTokens; j < end; ++j) {
    const int p = divide(j, a.cache.page);
    const int page = a.rows.table[it.s * a.rows.ld_table + p];
    if (page < 0 || page >= a.cache.num_pages) continue;
    const uint8_t *codes = a.cache.v + page * a.cache.page_stride +
                           it.h * a.cache.head_stride +
                           (j - p * a.cache.page_size) * a.cache.token_stride;
    for (int i = 0; i < 32 && k + i < a.cache.D; ++i)
      if (!Fm::finite(codes[k + i])) bad |= 1u << i;
  }
  return bad;
}

// mbar_wait by a whole warp, out of line: the kernel waits in many places.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                       unsigned *status, volatile int *abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, timeout_ns, status, abort_flag));
}

template <bool F32Q, int FMT, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_tc_kernel(const __grid_constant__ AttnArgs a, const uint64_t timeout_ns) {
  constexpr int TERMS = F32Q ? 2 : 1;
  using C = Cfg<DP, TERMS>;
  using Fm = Format<FMT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Share sh;
  __shared__ int64_t warp_sums[kThreads / 32];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + C::kBar;
  auto full_bar = [&](int i) { return bars + 8u * i; };                       // K or V
  auto empty_bar = [&](int i) { return bars + 8u * (C::SLOTS + i); };
  auto scfull_bar = [&](int i) { return bars + 8u * (2 * C::SLOTS + i); };    // scales
  auto scfree_bar = [&](int i) { return bars + 8u * (2 * C::SLOTS + kScaleBufs + i); };
  const uint32_t rest = bars + 8u * (2 * C::SLOTS + 2 * kScaleBufs);
  auto s_bar = [&](int t) { return rest + 8u * t; };         // scores are there
  auto p_bar = [&](int t, int half) { return rest + 8u * (2 + 2 * t + half); };  // weights
  auto pv_bar = [&](int t) { return rest + 8u * (6 + t); };  // O holds the first half's
  auto ofree_bar = [&](int t) { return rest + 8u * (8 + t); };
  auto factor_bar = [&](int i) { return rest + 8u * (10 + i); };
  auto fread_bar = [&](int i) { return rest + 8u * (12 + i); };
  const uint32_t qfull_bar = rest + 8u * 14, qempty_bar = rest + 8u * 15;
  const uint32_t done_bar = rest + 8u * 16;
  auto o_bar = [&](int t) { return rest + 8u * (17 + t); };  // O is an item's
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sbase + C::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + C::kMisc + 4);
  volatile int *poison = reinterpret_cast<volatile int *>(sbase + C::kMisc + 8);
  float *factors = reinterpret_cast<float *>(sbase + C::kFactors);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(full_bar(i), 4);
      mbar_init(empty_bar(i), 1);
    }
    for (int i = 0; i < kScaleBufs; ++i) {
      mbar_init(scfull_bar(i), 4);
      mbar_init(scfree_bar(i), 8);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_bar(t), 1);
      mbar_init(p_bar(t, 0), 4);
      mbar_init(p_bar(t, 1), 4);
      mbar_init(pv_bar(t), 1);
      mbar_init(o_bar(t), 1);
      mbar_init(ofree_bar(t), 4);
      mbar_init(factor_bar(t), kQWarps);
      mbar_init(fread_bar(t), 8);
    }
    mbar_init(qfull_bar, kQWarps);
    mbar_init(qempty_bar, 1);
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    *poison = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) a.desc[blockIdx.x].parts = 0;
  share_out<kThreads, kItemRows, kTokens>(a, &sh, warp_sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
           wait_long(bar, parity, timeout_ns, a.rows.status, abort_flag);
  };
  // Each warp's place in the work, in shared memory: registers are short.
  struct Place {
    Walk walk;
    Item it;
    int more;
  };
  __shared__ Place places[kThreads / 32];
  Place &my = places[warp];
  const Item &it = my.it;
  if (lane == 0) start_walk<kItemRows>(a, sh, &my.walk);
  auto next = [&] {
    __syncwarp();
    if (lane == 0) my.more = next_item<kItemRows, kTokens>(a, &my.walk, &my.it);
    __syncwarp();
    return my.more != 0;
  };

  if (warp < 8) {
    // --------------------------------------------------- scores to weights
    const int t = warp >> 2;                    // tile
    const int row = (warp & 3) * 32 + lane;     // of the tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_tm = lanes + C::kS + 128 * t, o_tm = lanes + C::kO + DP * t;
    uint32_t sc = 0;      // tiles of tokens so far
    uint32_t tiles = 0;   // those of them that this tile of rows took part in
    uint32_t items = 0;   // likewise
    bool ok = true;
    for (int n = 0; ok && next(); ++n) {
      const bool active = t * kRows < it.rows;
      const int r = it.rt * kItemRows + min(t * kRows + row, it.rows - 1);
      const int seen = t * kRows + row < it.rows ? tokens_seen(a, it.q, r) : 0;
      if (!(ok = wait(factor_bar(n & 1), (n >> 1) & 1u))) break;
      const float factor = factors[(n & 1) * kItemRows + t * kRows + row];
      const uint64_t factor2 = pair(factor, factor);
      __syncwarp();
      if (lane == 0) mbar_arrive(fread_bar(n & 1));
      float M = -INFINITY, back = 1.0f;  // back: what V's scales are relative to
      uint64_t l2 = pair(0.0f, 0.0f);
#pragma unroll 1
      for (int j = 0; j < it.count; ++j, ++sc) {
        const int buf = sc % kScaleBufs;
        if (!(ok = wait(scfull_bar(buf), (sc / kScaleBufs) & 1u))) break;
        if (!active) {
          if (lane == 0) mbar_arrive(scfree_bar(buf));
          continue;
        }
        const uint32_t scales = base + C::kScales + buf * kScaleBytes;
        if (j == 0) back = power_of_two(*reinterpret_cast<int *>(sbase + C::kScales + buf * kScaleBytes + 12 * kTokens));
        if (!(ok = wait(s_bar(t), tiles & 1u))) break;
        tc_fence_after();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          constexpr int HT = kTokens / 2;
          const uint32_t hs = scales + 4 * HT * half;
          float x[HT];
          tmem_load32(s_tm + HT * half, x);
          tmem_load32(s_tm + HT * half + 32, x + 32);
          tmem_wait32(x);
          tmem_wait32(x + 32);
#pragma unroll
          for (int i = 0; i < HT; i += 4) {
            uint64_t ks[2], lv[2];
            lds_pairs(hs + 4 * i, ks[0], ks[1]);
            lds_pairs(hs + 4 * kTokens + 4 * i, lv[0], lv[1]);
#pragma unroll
            for (int p = 0; p < 2; ++p)
              unpair(fma2(mul2(pair(x[i + 2 * p], x[i + 2 * p + 1]), ks[p]), factor2, lv[p]),
                     x[i + 2 * p], x[i + 2 * p + 1]);
          }
          const int limit = seen - (it.tile0 + j) * kTokens - HT * half;
          if (__any_sync(0xffffffffu, limit < HT)) {
#pragma unroll
            for (int i = 0; i < HT; ++i)
              if (i >= limit) x[i] = -INFINITY;
          }
          float best = x[0];
#pragma unroll
          for (int i = 1; i + 1 < HT; i += 2) best = max3(best, x[i], x[i + 1]);
          best = fmaxf(best, x[HT - 1]);
          if (__any_sync(0xffffffffu, best > M + kLazy)) {
            const float m = fmaxf(M, best);
            const float down = m == -INFINITY ? 1.0f : ex2(M - m);
            M = m;
            l2 = mul2(l2, pair(down, down));
            if (j > 0 || half > 0) {
              // The products of the tile before are in O, as the scores came after them.
              if (half > 0 && !(ok = wait(pv_bar(t), tiles & 1u))) break;
              tc_fence_after();
#pragma unroll 1
              for (int k = 0; k < DP; k += 32) {
                float o[32];
                tmem_load32(o_tm + k, o);
                tmem_wait32(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= down;
                tmem_store32(o_tm + k, o);
              }
            }
          }
          const float top = M == -INFINITY ? 0.0f : kShift - M;
          const uint64_t top2 = pair(top, top);
          uint64_t sum2 = pair(0.0f, 0.0f);
#pragma unroll
          for (int k = 0; k < HT; k += 32) {
            uint32_t w[16];
#pragma unroll
            for (int i = k; i < k + 32; i += 4) {
              uint64_t iv[2];
              lds_pairs(hs + 8 * kTokens + 4 * i, iv[0], iv[1]);
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                float u, v;
                unpair(add2(pair(x[i + 2 * p], x[i + 2 * p + 1]), top2), u, v);
                u = ex2(u);
                v = ex2(v);
                sum2 = fma2(pair(u, v), iv[p], sum2);
                w[(i - k) / 2 + p] = pack_half(u, v);
              }
            }
            tmem_store16(s_tm + (HT * half + k) / 2, w);
          }
          l2 = add2(l2, sum2);
          tmem_wait_store();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_bar(t, half));
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(scfree_bar(buf));
        ++tiles;
      }
      if (!ok) break;
      if (!active) continue;
      // The rows' results.
      if (!(ok = wait(o_bar(t), items & 1u))) break;
      ++items;
      tc_fence_after();
      float u, v;
      unpair(l2, u, v);
      const float sum = u + v;
      const bool some = sum > 0.0f || sum != sum;
      const float inv = some ? 1.0f / sum * back : 0.0f;
      const float lse = some ? M - kShift + log2f(sum) : -INFINITY;
      const bool mask = *poison != 0;
      const bool on = t * kRows + row < it.rows;
      const bool whole = it.count == it.tiles;
      const int part = 2 * blockIdx.x + (it.tile0 > 0 ? 0 : 1);
      const int tok = divide(r, a.group);
      const int64_t out_row = static_cast<int64_t>(it.q.row0) + tok;
      const int hq = it.h * a.G + r - tok * a.G;
      Weights weights = {1.0f, 0.0f, lse};
      if (whole && on) weights = weigh(a, out_row, hq, lse);
#pragma unroll 1
      for (int k = 0; k < DP; k += 32) {
        float o[32];
        tmem_load32(o_tm + k, o);
        tmem_wait32(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= inv;
        if (mask && on) {
          const uint32_t bad = lost_columns<Fm>(a, it, seen, k);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (bad >> i & 1u) o[i] = NAN;
        }
        if (on) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            if (k + i >= a.cache.D) break;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = o[i + e];
            if (whole) {
              emit<8>(a, out_row, hq, k + i, y, lse, weights);
            } else {
              float *p = a.part_o + (static_cast<int64_t>(part) * kItemRows + t * kRows + row) * DP + k + i;
              *reinterpret_cast<float4 *>(p) = make_float4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<float4 *>(p + 4) = make_float4(y[4], y[5], y[6], y[7]);
              if (k + i == 0) a.part_lse[part * kItemRows + t * kRows + row] = lse;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree_bar(t));
      if (threadIdx.x == 0 && !whole && it.tile0 == 0)
        a.desc[blockIdx.x] = {it.s, it.h, it.rt,
                              owner_of(sh, it.begin + it.tiles - 1) - static_cast<int>(blockIdx.x) + 1};
    }
  } else if (warp < 12) {
    // ------------------------------------------------- codes to halves
    // Three tiles of tokens are under way: of one the page numbers are being read, of
    // one the codes, and one is converted.  A warp has 16 tokens of each half of a tile,
    // a lane of which knows one, and reads back what it copied itself.
    const Cache &c = a.cache;
    constexpr int CH = DP / 16;        // 16-byte chunks of a row
    constexpr int PER = CH / 2;        // of a lane in a unit: 16 tokens of a warp
    const int tok0 = 16 * (warp - 8);
    const int token = (lane >> 4) * (kTokens / 2) + tok0 + (lane & 15);
    const uint32_t raw_at = base + C::kRaw + (warp - 8) * (C::kUnit / 4) + lane * 16;
    // The lane's chunk i of a unit.  Eight lanes cover even chunks of halves that are
    // swizzled by the token, so two tokens, one of them odd.
    const int ch = DP == 128 ? lane & 7 : lane & 3;
    auto local = [&](int i) {
      return DP == 128 ? (i >> 1) * 8 + (lane >> 3) * 2 + (((lane >> 2) & 1) ^ (i & 1))
                       : i * 8 + (lane >> 2);
    };
    // Peeked tile.
    bool peeked = false;
    int pj = 0, p_page = -1, p_page0 = -1, p_tok = 0, p_tok0 = 0;
    bool p_in = false, p_first = false, p_partial = false;
    int64_t p_head = 0, p_shead = 0;
    if (lane == 0) my.it.count = 0;
    __syncwarp();
    auto peek = [&] {
      if (pj == it.count) {
        peeked = next();
        pj = 0;
        if (!peeked) {
          if (lane == 0) my.it.count = 0;  // and it stays so
          __syncwarp();
          return;
        }
      }
      const int all = tokens_seen(a, it.q, it.rt * kItemRows);
      const int most = tokens_seen(a, it.q, it.rt * kItemRows + it.rows - 1);
      const int32_t *table = a.rows.table + it.s * a.rows.ld_table;
      p_first = pj == 0;
      p_tok0 = (it.tile0 + pj) * kTokens;
      p_tok = p_tok0 + token;
      p_in = p_tok < most;
      p_page = p_in ? table[divide(p_tok, c.page)] : -1;
      p_page0 = p_first && p_tok0 < most ? table[divide(p_tok0, c.page)] : -1;
      p_partial = p_tok0 + kTokens > all && all < most;
      p_head = it.h * c.head_stride;
      p_shead = it.h * c.scale_head_stride;
      ++pj;
    };
    // Located tile: where the lane's token is (-1: nowhere), its scales, and V's of the
    // item's first token.
    int64_t off = -1;
    float ks = 0.0f, vs = 1.0f, vs0 = 1.0f;
    bool located = false, first = false, partial = false;
    auto locate = [&] {
      located = peeked;
      if (!peeked) return;
      const bool good = p_in && p_page >= 0 && p_page < c.num_pages;
      if (p_in && !good) atomicOr(a.rows.status, kStatusBadDeviceArg);
      const int place = p_tok - divide(p_tok, c.page) * c.page_size;
      off = good ? p_page * c.page_stride + place * c.token_stride + p_head : -1;
      const int64_t so = p_page * c.scale_page_stride + place * c.scale_token_stride + p_shead;
      ks = good ? c.k_scale[so] : 0.0f;
      vs = good ? c.v_scale[so] : p_in ? NAN : 1.0f;
      first = p_first;
      partial = p_partial;
      vs0 = 1.0f;
      if (p_first && p_page0 >= 0 && p_page0 < c.num_pages)
        vs0 = c.v_scale[p_page0 * c.scale_page_stride +
                        (p_tok0 - divide(p_tok0, c.page) * c.page_size) * c.scale_token_stride +
                        p_shead];
    };
    // Unit `kind` (K, K, V, V) of the located tile.
    auto request = [&](int kind) {
      const uint8_t *from = kind < 2 ? c.k : c.v;
      const uint32_t dst = raw_at + kind % C::UNITS * C::kUnit;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int64_t o = __shfl_sync(0xffffffffu, off, (kind & 1) * 16 + local(i));
        const bool on = o >= 0 && ch * 16 < c.D;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * 512),
                     "l"(from + (on ? o + ch * 16 : 0)), "r"(on ? 16 : 0)
                     : "memory");
      }
    };
    int e0 = 0;
    uint32_t step = 0;                 // tiles of tokens
    bool ok = true;
    do {
      // The tile that is converted now, if any: its scales first.
      const bool cur = located, cur_partial = partial;
      if (cur) {
        if (first) e0 = exponent_of(vs0);
        const int buf = step % kScaleBufs;
        if (!(ok = wait(scfree_bar(buf), ((step / kScaleBufs) & 1u) ^ 1u))) break;
        float *scales = reinterpret_cast<float *>(sbase + C::kScales + buf * kScaleBytes);
        const bool fine = vs > 0.0f && vs < INFINITY;
        scales[token] = ks;
        scales[kTokens + token] = fine ? log2f(vs) - e0 : NAN;
        // A bad scale is in the exponent alone: rows that do not see it have weight 0.
        scales[2 * kTokens + token] =
            fine ? fminf(__fdiv_rn(power_of_two(e0), vs), 3.0e38f) : 1.0f;
        if (threadIdx.x == 8 * 32) *reinterpret_cast<int *>(scales + 3 * kTokens) = e0;
        __syncwarp();
        if (lane == 0) mbar_arrive(scfull_bar(buf));
      }
#pragma unroll 1
      for (int kind = 0; kind < 4; ++kind) {
        const uint32_t use = 2 * step + (kind >> 1);
        const int slot = use % C::SLOTS;
        if (kind == (C::UNITS == 4 ? 0 : 2)) {
          // With two units, V of this tile has been requested by now.
          locate();
          peek();
        }
        if (cur) {
          if ((kind & 1) == 0 &&
              !(ok = wait(empty_bar(slot), ((use / C::SLOTS) & 1u) ^ 1u)))
            break;
          asm volatile("cp.async.wait_group %0;" ::"n"(C::UNITS - 1) : "memory");
          const uint32_t src = raw_at + kind % C::UNITS * C::kUnit;
          const uint32_t dst = base + C::kRing + slot * C::kTileBytes + (ch >> 2) * C::kBlock;
          const bool clean = cur_partial && kind >= 2;
          bool found = false;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            uint32_t w[4], h[8];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(src + i * 512)
                         : "memory");
            if (clean) {
#pragma unroll
              for (int q = 0; q < 4; ++q) found |= Fm::clear4(w[q]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              h[2 * q] = decode2<FMT>(w[q] & 0xffffu);
              h[2 * q + 1] = decode2<FMT>(w[q] >> 16);
            }
            const uint32_t r = (kind & 1) * (kTokens / 2) + tok0 + local(i);
            const uint32_t row = dst + r * 128;
            const uint32_t c0 = 2 * (ch & 3), sw = r & 7;
            st_shared_v4(row + ((c0 ^ sw) << 4), h[0], h[1], h[2], h[3]);
            st_shared_v4(row + (((c0 + 1) ^ sw) << 4), h[4], h[5], h[6], h[7]);
          }
          if (found) *poison = 1;
        }
        const int ahead = (kind + C::UNITS) & 3;
        if (C::UNITS == 2 && kind < 2 ? cur : located) request(ahead);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (cur && (kind & 1)) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full_bar(slot));
        }
      }
      if (!ok) break;
      if (cur) ++step;
    } while (located || peeked);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else {
    if (warp == 12) {
      // ----------------------------------------------------------- MMAs
      constexpr uint32_t s_idesc = idesc_f16(kTokens, false), o_idesc = idesc_f16(DP, true);
      uint32_t s_step = 0, v_step = 0;      // tiles of tokens of S and of O
      uint32_t p_uses[2] = {0, 0}, o_uses[2] = {0, 0};
      // S of tile t against the K tile s_step.
      auto scores = [&](int t) {
        const uint32_t k = base + C::kRing + (2 * s_step) % C::SLOTS * C::kTileBytes;
#pragma unroll
        for (int term = 0; term < TERMS; ++term)
#pragma unroll
          for (int b = 0; b < DP / 64; ++b) {
            const uint64_t ad = smem_desc_k128_sw128(
                base + (t * TERMS + term) * C::kTileBytes + b * C::kBlock);
            const uint64_t bd = smem_desc_k128_sw128(k + b * C::kBlock);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              umma_ss(tmem + C::kS + 128 * t, ad + 2u * q, bd + 2u * q, s_idesc,
                      term > 0 || b > 0 || q > 0);
          }
        commit(s_bar(t));
      };
      auto k_ready = [&] {
        return wait(full_bar((2 * s_step) % C::SLOTS), ((2 * s_step) / C::SLOTS) & 1u);
      };
      bool ok = true, more = next();
      int rows = it.rows, count = it.count, n = 0;
      if (more) {
        ok = wait(qfull_bar, 0) && k_ready();
        if (ok) {
          tc_fence_after();
#pragma unroll 1
          for (int t = 0; t < 2; ++t)
            if (t * kRows < rows) scores(t);
          commit(empty_bar((2 * s_step) % C::SLOTS));
          if (count == 1) commit(qempty_bar);
          ++s_step;
        }
      }
      while (ok && more) {
        int next_rows = 0, next_count = 0;
#pragma unroll 1
        for (int j = 0; ok && j < count; ++j, ++v_step) {
          const bool last = j + 1 == count;
          if (last) {
            more = next();
            next_rows = more ? it.rows : 0;
            next_count = it.count;
          }
          const int s_rows = last ? next_rows : rows;
          const int v_slot = (2 * v_step + 1) % C::SLOTS;
          ok = wait(full_bar(v_slot), ((2 * v_step + 1) / C::SLOTS) & 1u);
          bool ready = false;
#pragma unroll 1
          for (int t = 0; ok && t < 2; ++t) {
            if (t * kRows < rows) {
              const uint32_t v = base + C::kRing + v_slot * C::kTileBytes;
#pragma unroll 1
              for (int half = 0; half < 2; ++half) {
                ok = wait(p_bar(t, half), (t ? p_uses[1] : p_uses[0]) & 1u);
                if (ok && j + half == 0 && (t ? o_uses[1] : o_uses[0]) > 0)
                  ok = wait(ofree_bar(t), ((t ? o_uses[1] : o_uses[0]) - 1) & 1u);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < kTokens / 32; ++q)
                  umma_ts(tmem + C::kO + DP * t, tmem + C::kS + 128 * t + 32 * half + 8 * q,
                          desc_mn(v + (half * (kTokens / 32) + q) * 2048, C::kBlock), o_idesc,
                          j > 0 || half > 0 || q > 0);
                if (half == 0) commit(pv_bar(t));
              }
              if (!ok) break;
              ++(t ? p_uses[1] : p_uses[0]);
              if (j == 0) ++(t ? o_uses[1] : o_uses[0]);
              if (last) commit(o_bar(t));
            }
            if (t * kRows < s_rows) {
              if (!ready) {
                if (last) ok = wait(qfull_bar, (n + 1) & 1u);
                ok = ok && k_ready();
                if (!ok) break;
                tc_fence_after();
                ready = true;
              }
              scores(t);
            }
          }
          if (!ok) break;
          commit(empty_bar(v_slot));
          if (s_rows > 0) {
            commit(empty_bar((2 * s_step) % C::SLOTS));
            if (last ? next_count == 1 : j + 2 == count) commit(qempty_bar);
            ++s_step;
          }
        }
        rows = next_rows;
        count = next_count;
        ++n;
      }
      commit(done_bar);
      mbar_wait_drain(done_bar, 0, timeout_ns, a.rows.status);
    } else {
      // -------------------------------------------------------- query rows
      constexpr int LR = DP / 8;          // lanes of a row, 8 elements each
      constexpr int RP = 32 / LR;         // rows of a pass
      const int sub = lane % LR;
      const bool vec = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0 &&
                       (a.ldq * (F32Q ? 4 : 2)) % 16 == 0 &&
                       (a.ldq_head * (F32Q ? 4 : 2)) % 16 == 0;
      for (int n = 0; next(); ++n) {
        // q's rows are in use until the scores of the item before are done, its
        // factors (two items' worth) until every warp has read them.
        if (!wait(qempty_bar, (n & 1u) ^ 1u) || !wait(fread_bar(n & 1), ((n >> 1) & 1u) ^ 1u))
          break;
        auto place = [&](int rr, int term) {
          const int t = rr / kRows, row = rr % kRows;
          return base + (t * TERMS + term) * C::kTileBytes + (sub / 8) * C::kBlock + row * 128 +
                 (((sub & 7) ^ (row & 7)) << 4);
        };
        const int rows = it.rows > kRows ? kItemRows : kRows;
        constexpr int kPass = RP * kQWarps;     // rows of a pass of all three warps
        const int r_first = RP * (warp - 13) + lane / LR;
#pragma unroll 2
        for (int rr = r_first; rr < rows; rr += kPass) {
          const bool on = rr < it.rows && 8 * sub < a.cache.D;
          const int r = it.rt * kItemRows + min(rr, it.rows - 1);
          const int tok = divide(r, a.group);
          const int64_t at = (static_cast<int64_t>(it.q.row0) + tok) * a.ldq +
                             (it.h * a.G + r - tok * a.G) * a.ldq_head + 8 * sub;
          if (vec || !on) {
#pragma unroll
            for (int term = 0; term < TERMS; ++term) {
              const uint8_t *from = static_cast<const uint8_t *>(a.q) +
                                    (on ? at * (F32Q ? 4 : 2) + 16 * term : 0);
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(place(rr, term)),
                           "l"(vec ? from : reinterpret_cast<const uint8_t *>(a.cache.k)),
                           "r"(on ? 16 : 0)
                           : "memory");
            }
          } else if (F32Q) {
            const uint32_t *p = static_cast<const uint32_t *>(a.q) + at;
            st_shared_v4(place(rr, 0), p[0], p[1], p[2], p[3]);
            st_shared_v4(place(rr, TERMS - 1), p[4], p[5], p[6], p[7]);
          } else {
            const uint16_t *p = static_cast<const uint16_t *>(a.q) + at;
            st_shared_v4(place(rr, 0), p[0] | p[1] << 16, p[2] | p[3] << 16,
                         p[4] | p[5] << 16, p[6] | p[7] << 16);
          }
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        // Four rows of a lane at a time, so that their steps overlap.
#pragma unroll 1
        for (int r0 = r_first; r0 - lane / LR < rows; r0 += 4 * kPass) {
          uint32_t w[4][TERMS][4];
          float m[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int rr = r0 + u * kPass;
            m[u] = 0.0f;
#pragma unroll
            for (int term = 0; term < TERMS; ++term) {
              w[u][term][0] = w[u][term][1] = w[u][term][2] = w[u][term][3] = 0;
              if (rr < rows)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[u][term][0]), "=r"(w[u][term][1]), "=r"(w[u][term][2]),
                               "=r"(w[u][term][3])
                             : "r"(place(rr, term))
                             : "memory");
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t b = w[u][term][i];
                if (F32Q) {
                  m[u] = fmaxf(m[u], fabsf(__uint_as_float(b)));
                } else {
                  m[u] = fmaxf(m[u], fabsf(__uint_as_float(b << 16)));
                  m[u] = fmaxf(m[u], fabsf(__uint_as_float(b & 0xffff0000u)));
                }
              }
            }
          }
#pragma unroll
          for (int o = LR / 2; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int rr = r0 + u * kPass;
            if (rr >= rows) continue;
            const int e = min(max(8 - exponent_of(m[u]), -126), 126);
            const float up = power_of_two(e);
            uint32_t h[TERMS][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x, y;
              if (F32Q) {  // elements 2 i, 2 i + 1
                x = __uint_as_float(w[u][TERMS == 2 ? i >> 1 : 0][2 * (i & 1)]) * up;
                y = __uint_as_float(w[u][TERMS == 2 ? i >> 1 : 0][2 * (i & 1) + 1]) * up;
              } else {
                x = __uint_as_float(w[u][0][i] << 16) * up;
                y = __uint_as_float(w[u][0][i] & 0xffff0000u) * up;
              }
              h[0][i] = pack_half(x, y);
              if (TERMS == 2) {
                const float2 f = half2_floats(h[0][i]);
                h[TERMS - 1][i] = pack_half(x - f.x, y - f.y);
              }
            }
#pragma unroll
            for (int term = 0; term < TERMS; ++term)
              st_shared_v4(place(rr, term), h[term][0], h[term][1], h[term][2], h[term][3]);
            if (sub == 0)
              factors[(n & 1) * kItemRows + rr] = power_of_two(-e) * a.scale_log2;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(factor_bar(n & 1));
          mbar_arrive(qfull_bar);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool F32Q, int FMT, int DP>
fp8la_status launch_one(const AttnArgs &a, int slot, int ctas, cudaStream_t s) {
  using C = Cfg<DP, F32Q ? 2 : 1>;
  auto kern = kv_attention_tc_kernel<F32Q, FMT, DP>;
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::kAlloc);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kAlloc;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, wait_timeout_ns()) == cudaSuccess ? FP8LA_OK
                                                                             : FP8LA_ERR_CUDA;
}

}  // namespace

fp8la_status launch_many(const AttnArgs &a, bool f32, int format, int ctas, cudaStream_t s) {
  const int which = (f32 ? 4 : 0) | (format == FP8LA_FORMAT_E5M2 ? 2 : 0) | (a.cache.D > 64);
  switch (which) {
    case 0: return launch_one<false, 0, 64>(a, 92, ctas, s);
    case 1: return launch_one<false, 0, 128>(a, 93, ctas, s);
    case 2: return launch_one<false, 1, 64>(a, 94, ctas, s);
    case 3: return launch_one<false, 1, 128>(a, 95, ctas, s);
    case 4: return launch_one<true, 0, 64>(a, 96, ctas, s);
    case 5: return launch_one<true, 0, 128>(a, 97, ctas, s);
    case 6: return launch_one<true, 1, 64>(a, 98, ctas, s);
    default: return launch_one<true, 1, 128>(a, 99, ctas, s);
  }
}

}  // namespace kv
}  // namespace fp8la

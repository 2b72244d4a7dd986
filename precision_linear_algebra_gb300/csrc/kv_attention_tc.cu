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
// Registers of a thread of each role; the launch gives every thread 128.
constexpr int kSoftmaxRegs = 176, kConvertRegs = 104, kOtherRegs = 56;
static_assert(2 * kSoftmaxRegs + kConvertRegs + kOtherRegs <= 4 * 128, "registers");

template <int DP, int TERMS>
struct Cfg {
  static constexpr int kBlock = kRows * 128;            // 64 elements of each row
  static constexpr int kTileBytes = DP / 64 * kBlock;   // halves of a tile
  static constexpr int kQ = 2 * TERMS * kTileBytes;
  static constexpr int SLOTS = kQ + 4 * kTileBytes <= 200 * 1024 ? 4 : 2;
  static constexpr int kRing = kQ;
  static constexpr int kScales = kRing + SLOTS * kTileBytes;
  static constexpr int kFactors = kScales + kScaleBufs * kScaleBytes;
  static constexpr int kBar = kFactors + 2 * kItemRows * 4;
  static constexpr int kBars = 2 * SLOTS + 2 * kScaleBufs + 15;
  static constexpr int kMisc = kBar + kBars * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static constexpr int kS = 0, kO = 256;                // tensor memory columns
  static_assert(kAlloc <= 226 * 1024, "shared memory");
  static_assert(kO + 2 * DP <= 512, "tensor memory");
};

// D[tmem] (+)= A B^T, halves, FP32 sums; A from shared memory, or from tensor memory.
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
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

template <int N>
__device__ __forceinline__ void set_more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ int exponent_of(float v) {
  const int e = static_cast<int>(__float_as_uint(v) >> 23);
  if (v == 0.0f || e >= 255) return 0;
  return e > 0 ? e - 127 : -126;
}
__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// One item's part that this CTA goes through.
struct Item {
  Seq q;
  int s, h, rt, tile0, count, tiles, rows;  // rows: of the item, up to 256
  int64_t begin;                            // its first unit, of all
};

// Walks through this CTA's items; every role does so for itself.
struct Walk {
  int64_t at, before;
  int s;
  __device__ bool next(const AttnArgs &a, const Share &sh, Item &it) {
    if (at >= sh.end) return false;
    Seq q = load_seq(a, s);
    int64_t units = units_of<kItemRows, kTokens, true>(a, q);
    while (at >= before + units * a.cache.heads) {
      before += units * a.cache.heads;
      q = load_seq(a, ++s);
      units = units_of<kItemRows, kTokens, true>(a, q);
    }
    const int64_t local = at - before;
    it.h = static_cast<int>(local / units);
    int64_t left = local - it.h * units;
    int rt = 0, n = tiles_of<kItemRows, kTokens, true>(a, q, 0);
    while (left >= n) {
      left -= n;
      n = tiles_of<kItemRows, kTokens, true>(a, q, ++rt);
    }
    it.q = q;
    it.s = s;
    it.rt = rt;
    it.tile0 = static_cast<int>(left);
    it.tiles = n;
    it.begin = at - left;
    it.count = static_cast<int>(min(static_cast<int64_t>(n - it.tile0), sh.end - at));
    it.rows = min(kItemRows, q.n * a.G - rt * kItemRows);
    at += it.count;
    return true;
  }
};

template <bool F32Q, int FMT, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_tc_kernel(const AttnArgs a, const uint64_t timeout_ns) {
  constexpr int TERMS = F32Q ? 2 : 1;
  using C = Cfg<DP, TERMS>;
  using Fm = Format<FMT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Share share_slot;
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
  auto p_bar = [&](int t) { return rest + 8u * (2 + t); };   // weights are
  auto pv_bar = [&](int t) { return rest + 8u * (4 + t); };  // O holds their products
  auto ofree_bar = [&](int t) { return rest + 8u * (6 + t); };
  auto factor_bar = [&](int i) { return rest + 8u * (8 + i); };
  auto fread_bar = [&](int i) { return rest + 8u * (10 + i); };
  const uint32_t qfull_bar = rest + 8u * 12, qempty_bar = rest + 8u * 13;
  const uint32_t done_bar = rest + 8u * 14;
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
      mbar_init(p_bar(t), 4);
      mbar_init(pv_bar(t), 1);
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
  const Share sh = share_out<kThreads, kItemRows, kTokens, true>(a, &share_slot, warp_sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu,
                      mbar_wait(bar, parity, timeout_ns, a.rows.status, abort_flag));
  };
  Walk walk{sh.begin, sh.before, sh.seq};
  Item it;

  if (warp < 8) {
    // --------------------------------------------------- scores to weights
    set_more_regs<kSoftmaxRegs>();
    const int t = warp >> 2;                    // tile
    const int row = (warp & 3) * 32 + lane;     // of the tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_tm = lanes + C::kS + 128 * t, o_tm = lanes + C::kO + DP * t;
    uint32_t sc = 0;      // tiles of tokens so far
    uint32_t mine = 0;    // those of them that this tile of rows took part in
    bool ok = true;
    for (int n = 0; ok && walk.next(a, sh, it); ++n) {
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
        if (!(ok = wait(s_bar(t), mine & 1u))) break;
        tc_fence_after();
        float x[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; k += 32) tmem_load32(s_tm + k, x + k);
        float best = -INFINITY;
#pragma unroll
        for (int k = 0; k < kTokens; k += 32) {
          tmem_wait32(x + k);
#pragma unroll
          for (int i = k; i < k + 32; i += 4) {
            uint64_t ks[2], lv[2];
            lds_pairs(scales + 4 * i, ks[0], ks[1]);
            lds_pairs(scales + 4 * kTokens + 4 * i, lv[0], lv[1]);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint64_t v = fma2(mul2(pair(x[i + 2 * p], x[i + 2 * p + 1]), ks[p]),
                                      factor2, lv[p]);
              unpair(v, x[i + 2 * p], x[i + 2 * p + 1]);
            }
          }
        }
        const int limit = seen - (it.tile0 + j) * kTokens;
        const bool edge = __any_sync(0xffffffffu, limit < kTokens);
        if (edge) {
#pragma unroll
          for (int i = 0; i < kTokens; ++i)
            if (i >= limit) x[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < kTokens; i += 2) best = fmaxf(best, fmaxf(x[i], x[i + 1]));
        if (__any_sync(0xffffffffu, best > M + kLazy)) {
          const float m = fmaxf(M, best);
          const float down = m == -INFINITY ? 1.0f : ex2(M - m);
          M = m;
          l2 = mul2(l2, pair(down, down));
          if (j > 0) {
            if (!(ok = wait(pv_bar(t), (mine - 1) & 1u))) break;
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
        for (int k = 0; k < kTokens; k += 32) {
          uint32_t w[16];
#pragma unroll
          for (int i = k; i < k + 32; i += 4) {
            uint64_t iv[2];
            lds_pairs(scales + 8 * kTokens + 4 * i, iv[0], iv[1]);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              float u, v;
              unpair(add2(pair(x[i + 2 * p], x[i + 2 * p + 1]), top2), u, v);
              u = ex2(u);
              v = ex2(v);
              if (edge) {
                // 1 / vs of a token that the row does not see may be anything.
                float du, dv;
                unpair(iv[p], du, dv);
                if (x[i + 2 * p] == -INFINITY) du = 0.0f;
                if (x[i + 2 * p + 1] == -INFINITY) dv = 0.0f;
                iv[p] = pair(du, dv);
              }
              sum2 = fma2(pair(u, v), iv[p], sum2);
              w[(i - k) / 2 + p] = pack_half(u, v);
            }
          }
          tmem_store16(s_tm + k / 2, w);
        }
        l2 = add2(l2, sum2);
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_bar(t));
          mbar_arrive(scfree_bar(buf));
        }
        ++mine;
      }
      if (!ok) break;
      if (!active) continue;
      // The rows' results.
      if (!(ok = wait(pv_bar(t), (mine - 1) & 1u))) break;
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
      const int all = tokens_seen(a, it.q, it.rt * kItemRows);
#pragma unroll 1
      for (int k = 0; k < DP; k += 32) {
        float o[32];
        tmem_load32(o_tm + k, o);
        tmem_wait32(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= inv;
        if (mask && on) {
          // Codes that are not finite, of the tiles that were written without them.
          const int end = min(seen, (it.tile0 + it.count) * kTokens);
          for (int j = max(it.tile0 * kTokens, all / kTokens * kTokens); j < end; ++j) {
            const int p = divide(j, a.cache.page);
            const int page = a.rows.table[it.s * a.rows.ld_table + p];
            if (page < 0 || page >= a.cache.num_pages) continue;
            const uint8_t *codes = a.cache.v + page * a.cache.page_stride +
                                   it.h * a.cache.head_stride +
                                   (j - p * a.cache.page_size) * a.cache.token_stride;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (k + i < a.cache.D && !Fm::finite(codes[k + i])) o[i] = NAN;
          }
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
    set_fewer_regs<kConvertRegs>();
    const Cache &c = a.cache;
    constexpr int CH = DP / 16;        // 16-byte chunks of a row
    constexpr int PER = CH;            // chunks of a lane: 32 tokens of a warp
    const int tok0 = 32 * (warp - 8);
    uint32_t step = 0;                 // tiles of tokens
    bool ok = true;
    uint4 kb[PER], vb[PER];
    for (int n = 0; ok && walk.next(a, sh, it); ++n) {
      const int64_t head = it.h * c.head_stride;
      const int64_t shead = it.h * c.scale_head_stride;
      const int all = tokens_seen(a, it.q, it.rt * kItemRows);
      const int most = tokens_seen(a, it.q, it.rt * kItemRows + it.rows - 1);
      const int32_t *table = a.rows.table + it.s * a.rows.ld_table;
      // Lane's token of tile j: where its codes are (-1: nowhere), and its scales.
      auto page_of = [&](int j) {
        const int tk = (it.tile0 + j) * kTokens + tok0 + lane;
        return j < it.count && tk < most ? table[divide(tk, c.page)] : -1;
      };
      int page = page_of(0);
      int64_t off;
      float ks, vs;
      auto locate = [&](int j) {
        const int tk = (it.tile0 + j) * kTokens + tok0 + lane;
        const bool in = j < it.count && tk < most;
        const bool good = in && page >= 0 && page < c.num_pages;
        if (in && !good) atomicOr(a.rows.status, kStatusBadDeviceArg);
        const int place = tk - divide(tk, c.page) * c.page_size;
        off = good ? page * c.page_stride + place * c.token_stride + head : -1;
        const int64_t so = page * c.scale_page_stride + place * c.scale_token_stride + shead;
        ks = good ? c.k_scale[so] : 0.0f;
        vs = good ? c.v_scale[so] : in ? NAN : 1.0f;
      };
      auto load = [&](const uint8_t *from, uint4 (&b)[PER]) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int id = lane + 32 * i, token = id / CH, ch = id % CH;
          const int64_t o = __shfl_sync(0xffffffffu, off, token);
          b[i] = make_uint4(0, 0, 0, 0);
          if (o >= 0 && ch * 16 < c.D)
            b[i] = *reinterpret_cast<const uint4 *>(from + o + ch * 16);
        }
      };
      auto write = [&](uint32_t dst, const uint4 (&b)[PER]) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int id = lane + 32 * i, token = tok0 + id / CH, ch = id % CH;
          const uint32_t w[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
          uint32_t h[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            h[2 * q] = decode2<FMT>(w[q] & 0xffffu);
            h[2 * q + 1] = decode2<FMT>(w[q] >> 16);
          }
          const uint32_t row = dst + (ch >> 2) * C::kBlock + token * 128;
          const uint32_t c0 = 2 * (ch & 3), sw = token & 7;
          // Lanes of the second block of columns begin with their second half, so
          // that eight lanes write to eight different banks of 16 bytes.
          const bool flip = (ch & 4) != 0;
          const uint32_t first = row + (((c0 + (flip ? 1 : 0)) ^ sw) << 4);
          const uint32_t second = row + (((c0 + (flip ? 0 : 1)) ^ sw) << 4);
          st_shared_v4(first, flip ? h[4] : h[0], flip ? h[5] : h[1], flip ? h[6] : h[2],
                       flip ? h[7] : h[3]);
          st_shared_v4(second, flip ? h[0] : h[4], flip ? h[1] : h[5], flip ? h[2] : h[6],
                       flip ? h[3] : h[7]);
        }
      };
      locate(0);
      page = page_of(1);
      load(c.k, kb);
      // V's scales are taken relative to a power of two near that of the first token.
      int e0 = 0;
      if (it.tile0 * kTokens < most) {
        const int tk = it.tile0 * kTokens, p = divide(tk, c.page), pg = table[p];
        if (pg >= 0 && pg < c.num_pages)
          e0 = exponent_of(c.v_scale[pg * c.scale_page_stride +
                                     (tk - p * c.page_size) * c.scale_token_stride + shead]);
      }
#pragma unroll 1
      for (int j = 0; j < it.count; ++j, ++step) {
        load(c.v, vb);
        // Scales, then K.
        const int buf = step % kScaleBufs;
        if (!(ok = wait(scfree_bar(buf), ((step / kScaleBufs) & 1u) ^ 1u))) break;
        float *scales = reinterpret_cast<float *>(sbase + C::kScales + buf * kScaleBytes);
        const bool fine = vs > 0.0f && vs < INFINITY;
        scales[tok0 + lane] = ks;
        scales[kTokens + tok0 + lane] = fine ? log2f(vs) - e0 : NAN;
        scales[2 * kTokens + tok0 + lane] = fine ? __fdiv_rn(power_of_two(e0), vs) : NAN;
        if (threadIdx.x == 8 * 32) *reinterpret_cast<int *>(scales + 3 * kTokens) = e0;
        __syncwarp();
        if (lane == 0) mbar_arrive(scfull_bar(buf));
        const uint32_t k_use = 2 * step, v_use = 2 * step + 1;
        const int k_slot = k_use % C::SLOTS, v_slot = v_use % C::SLOTS;
        if (!(ok = wait(empty_bar(k_slot), ((k_use / C::SLOTS) & 1u) ^ 1u))) break;
        write(base + C::kRing + k_slot * C::kTileBytes, kb);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full_bar(k_slot));
        // The next tile's K is under way while V is written.
        locate(j + 1);
        page = page_of(j + 2);
        load(c.k, kb);
        // Tokens that some row of the item does not see.
        if ((it.tile0 + j + 1) * kTokens > all && all < most) {
          bool found = false;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            uint32_t *w = reinterpret_cast<uint32_t *>(&vb[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int b = 0; b < 4; ++b)
                if (!Fm::finite(w[q] >> (8 * b))) {
                  w[q] &= ~(0xffu << (8 * b));
                  found = true;
                }
          }
          if (found) *poison = 1;
        }
        if (!(ok = wait(empty_bar(v_slot), ((v_use / C::SLOTS) & 1u) ^ 1u))) break;
        write(base + C::kRing + v_slot * C::kTileBytes, vb);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full_bar(v_slot));
      }
    }
  } else {
    set_fewer_regs<kOtherRegs>();
    if (warp == 12) {
      // ----------------------------------------------------------- MMAs
      constexpr uint32_t s_idesc = idesc_f16(kTokens, false), o_idesc = idesc_f16(DP, true);
      if (lane == 0) {
        uint32_t s_step = 0, v_step = 0;      // tiles of tokens of S and of O
        uint32_t p_uses[2] = {0, 0}, o_uses[2] = {0, 0};
        auto await = [&](uint32_t bar, uint32_t parity) {
          return mbar_wait(bar, parity, timeout_ns, a.rows.status, abort_flag);
        };
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
          umma_commit(s_bar(t));
        };
        auto k_ready = [&] {
          return await(full_bar((2 * s_step) % C::SLOTS), ((2 * s_step) / C::SLOTS) & 1u);
        };
        bool ok = true, more = walk.next(a, sh, it);
        int n = 0;
        if (more) {
          ok = await(qfull_bar, 0) && k_ready();
          if (ok) {
            tc_fence_after();
            for (int t = 0; t < 2; ++t)
              if (t * kRows < it.rows) scores(t);
            umma_commit(empty_bar((2 * s_step) % C::SLOTS));
            if (it.count == 1) umma_commit(qempty_bar);
            ++s_step;
          }
        }
        while (ok && more) {
          Item next;
          bool have = false;
          for (int j = 0; ok && j < it.count; ++j, ++v_step) {
            const bool last = j + 1 == it.count;
            if (last) have = walk.next(a, sh, next);
            const int rows = last ? (have ? next.rows : 0) : it.rows;
            const int v_slot = (2 * v_step + 1) % C::SLOTS;
            ok = await(full_bar(v_slot), ((2 * v_step + 1) / C::SLOTS) & 1u);
            bool ready = false;
            for (int t = 0; ok && t < 2; ++t) {
              if (t * kRows < it.rows) {
                ok = await(p_bar(t), p_uses[t] & 1u);
                if (ok && j == 0 && o_uses[t] > 0) ok = await(ofree_bar(t), (o_uses[t] - 1) & 1u);
                if (!ok) break;
                ++p_uses[t];
                if (j == 0) ++o_uses[t];
                tc_fence_after();
                const uint32_t v = base + C::kRing + v_slot * C::kTileBytes;
#pragma unroll
                for (int q = 0; q < kTokens / 16; ++q)
                  umma_ts(tmem + C::kO + DP * t, tmem + C::kS + 128 * t + 8 * q,
                          desc_mn(v + q * 2048, C::kBlock), o_idesc, j > 0 || q > 0);
                umma_commit(pv_bar(t));
              }
              if (t * kRows < rows) {
                if (!ready) {
                  if (last) ok = await(qfull_bar, (n + 1) & 1u);
                  ok = ok && k_ready();
                  if (!ok) break;
                  tc_fence_after();
                  ready = true;
                }
                scores(t);
              }
            }
            if (!ok) break;
            umma_commit(empty_bar(v_slot));
            if (rows > 0) {
              umma_commit(empty_bar((2 * s_step) % C::SLOTS));
              if (last ? next.count == 1 : j + 2 == it.count) umma_commit(qempty_bar);
              ++s_step;
            }
          }
          if (!ok) break;
          it = next;
          more = have;
          ++n;
        }
        umma_commit(done_bar);
        mbar_wait_drain(done_bar, 0, timeout_ns, a.rows.status);
      }
    } else {
      // -------------------------------------------------------- query rows
      constexpr int LR = DP / 8;          // lanes of a row, 8 elements each
      constexpr int RP = 32 / LR;         // rows of a pass
      const int sub = lane % LR;
      const bool vec = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0 &&
                       (a.ldq * (F32Q ? 4 : 2)) % 16 == 0 &&
                       (a.ldq_head * (F32Q ? 4 : 2)) % 16 == 0;
      for (int n = 0; walk.next(a, sh, it); ++n) {
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
        for (int r0 = RP * (warp - 13); r0 < rows; r0 += RP * kQWarps) {
          const int rr = r0 + lane / LR;
          if (rr >= rows) continue;
          const bool on = rr < it.rows && 8 * sub < a.cache.D;
          const int r = it.rt * kItemRows + min(rr, it.rows - 1);
          const int tok = divide(r, a.group);
          const int64_t at = (static_cast<int64_t>(it.q.row0) + tok) * a.ldq +
                             (it.h * a.G + r - tok * a.G) * a.ldq_head + 8 * sub;
          if (vec || !on) {
#pragma unroll
            for (int term = 0; term < TERMS; ++term) {
              const void *from = F32Q ? static_cast<const void *>(static_cast<const float *>(a.q) + (on ? at + 4 * term : 0))
                                      : static_cast<const void *>(static_cast<const uint16_t *>(a.q) + (on ? at : 0));
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(place(rr, term)),
                           "l"(vec ? from : static_cast<const void *>(a.out)), "r"(on ? 16 : 0)
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
        for (int r0 = RP * (warp - 13); r0 < rows; r0 += RP * kQWarps) {
          const int rr = r0 + lane / LR;
          const bool in = rr < rows;
          const uint32_t p0 = place(in ? rr : 0, 0), p1 = place(in ? rr : 0, TERMS - 1);
          uint32_t w[2][4] = {};
          float x[8];
          if (in) {
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0][0]), "=r"(w[0][1]), "=r"(w[0][2]), "=r"(w[0][3])
                         : "r"(p0) : "memory");
            if (F32Q)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[1][0]), "=r"(w[1][1]), "=r"(w[1][2]), "=r"(w[1][3])
                           : "r"(p1) : "memory");
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[i] = F32Q ? __uint_as_float(w[i >> 2][i & 3])
                        : __uint_as_float(i & 1 ? w[0][i >> 1] & 0xffff0000u : w[0][i >> 1] << 16);
          float m = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
          for (int o = LR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const int e = min(max(8 - exponent_of(m), -126), 126);
          const float up = power_of_two(e);
          if (in) {
#pragma unroll
            for (int term = 0; term < TERMS; ++term) {
              uint32_t h[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (term == 0) {
                  x[2 * i] *= up;
                  x[2 * i + 1] *= up;
                }
                h[i] = pack_half(x[2 * i], x[2 * i + 1]);
                const float2 f = half2_floats(h[i]);
                x[2 * i] -= f.x;
                x[2 * i + 1] -= f.y;
              }
              st_shared_v4(term == 0 ? p0 : p1, h[0], h[1], h[2], h[3]);
            }
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
        cudaFuncAttributes f;
        cudaError_t e = cudaFuncGetAttributes(&f, kern);
        // The roles' registers come out of the launch's; too few would never arrive.
        if (e == cudaSuccess && f.numRegs != 128) e = cudaErrorInvalidConfiguration;
        return e != cudaSuccess
                   ? e
                   : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
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

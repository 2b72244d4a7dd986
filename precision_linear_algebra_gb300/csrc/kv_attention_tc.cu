// Attention of many rows over the FP8 key/value cache, on the 5th-generation tensor
// cores.  Formulas and precision as in kv_attention.cu.
//
// Bound: the tensor cores at the half rate (q and the weights are not quantised to
// FP8), and beside them the exponentials and the conversions.  A CTA takes 256 rows,
// two tiles of 128, against tiles of 128 tokens, so that one tile's products run
// while the other's weights are made:
//
//   warps 0-3, 4-7   a tile of rows each: scores from tensor memory, running maximum,
//                    weights as halves back over them; before that the tile's rows of q,
//                    scaled by a power of two to halves (an FP32 row as two terms), in
//                    place over what cp.async brought while the last tile of the rows
//                    before was at work
//   warps 8-12       codes from the cache (16 bytes a copy) to halves in shared memory,
//                    swizzled as the MMA reads them, 16 tokens of K or V at a time; V is
//                    read as the transposed operand
//   warps 13, 14     where the tokens lie (any pages), K's scales and V's, and which tokens
//                    have shares of the denominator that are added up beside (see kSpan),
//                    rows of zeros in V among them
//   warp 15          issues the MMAs: S = Q K^T from shared memory, O += P V with P in
//                    tensor memory
//
// Four warps an SM partition do four different things, so what bounds the loops is
// first of all the fetching of their instructions: they are kept short (the first
// version's unrolled ones did not fit the instruction cache and took 863 us instead of
// what is below).
//
// Measured, 8 K/V heads of 128, 8 query heads each, us and TFLOP/s of what is visible:
// two prompts of 2048 tokens 264 (520; this kernel 250), one of 8192 1379 (797), 512
// rows after 32768 tokens 638 (868), 4096 FP32 rows 572 (481: two terms, twice the
// scores' products).  A tile of 256 rows and 128 tokens takes 3 us, 1.3 of them on the
// tensor cores; the rest is the chain from scores to weights in 8 warps (64 registers of
// scores each, 1.9 instructions a cycle and SM), and an item's rows of q and of O are
// not hidden behind it, which is what kItemCost counts.
//
// Tensor memory: S (and P over it) and O of both tiles, 512 columns with D = 128.
// O stays there; a row's is rescaled only where its maximum grew by 2^8.  A part of more
// than kPiece tiles goes through in pieces, as the tensor cores cut what they add.
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
constexpr int kItemRows = kManyItemRows;
constexpr int kTokens = kTileTokens;
// What an item costs beside its tiles, in tiles: bringing its rows, writing them out.
// Two prompts of 2048 tokens, us, with 2, 3, 4: 273, 267, 273.
constexpr int kItemCost = kManyItemCost;
constexpr int kItemBufs = 4;
constexpr int kItemReaders = 10;    // the warps that make weights, 14 and 15
constexpr int kConverters = 5;
constexpr int kGroup = 16;          // tokens of a converter's job
constexpr int kJobs = 2 * kTokens / kGroup;  // of a tile, K's first
// K's scales, log2 and reciprocal of V's, and of the tile: the exponent that V's are relative
// to, whether it rose (1) and whether there are tokens whose shares are added up beside (2),
// by how much it rose, and, from the fifth word on, those tokens' bits (see kSpan).
constexpr int kScaleBufs = 4;
constexpr int kTileHead = 3 * kTokens * 4;
constexpr int kScaleBytes = kTileHead + 32;
constexpr float kShift = 7.0f;      // as in kv_attention.cu
constexpr float kLazy = 8.0f;
template <int DP, int TERMS>
struct Cfg {
  static constexpr int kBlock = kRows * 128;            // 64 elements of each row
  static constexpr int kTileBytes = DP / 64 * kBlock;   // halves of a tile
  static constexpr int kQ = 2 * TERMS * kTileBytes;
  static constexpr int SLOTS = TERMS == 1 ? 3 : 2;      // K's and V's tiles in turn
  static constexpr int kRing = kQ;
  // Jobs of a converter whose codes are under way.
  static constexpr int AHEAD = TERMS == 1 ? 3 : 1;
  static constexpr int kJob = kGroup * DP;
  static constexpr int kRaw = kRing + SLOTS * kTileBytes;
  static constexpr int kPlaces = kRaw + kConverters * AHEAD * kJob;
  static constexpr int kScales = kPlaces + kScaleBufs * kTokens * 8;
  static constexpr int kFactors = kScales + kScaleBufs * kScaleBytes;
  static constexpr int kFirst = kFactors + kItemRows * 4;  // 16 codes of each row of V, two tiles
  static constexpr int kBar = kFirst + 2 * kTokens * 16;
  static constexpr int kBars = 2 * SLOTS + 4 * kScaleBufs + 14 + 2 * kItemBufs;
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

// 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
        "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]),
        "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
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
// 16 lanes of 64 columns: registers 4 i + {0, 1} hold this thread's row (lane / 4) in
// columns 8 i + 2 (lane % 4) + {0, 1}, registers 4 i + {2, 3} the row 8 further.
__device__ __forceinline__ void tmem_load_rows(uint32_t addr, float *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
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
// The same of 32 columns; the load waits.
__device__ __forceinline__ void tmem_load_rows16(uint32_t addr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
        "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]),
        "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store_rows16(uint32_t addr, const float (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      ::"f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]),
        "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]),
        "f"(r[14]), "f"(r[15]), "r"(addr)
      : "memory");
}
// 16 lanes of 32 columns, a pair of halves each: registers 2 i and 2 i + 1 hold columns
// 4 i + lane % 4 of the rows lane / 4 and 8 further.
__device__ __forceinline__ void tmem_store_halves(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
// 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_store16(uint32_t addr, const float (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      ::"f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]),
        "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]),
        "f"(r[14]), "f"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 32 bytes, 32-byte aligned: a row's whole sector at once.
__device__ __forceinline__ void store32(void *p, const uint32_t (&u)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

// A condition that is the same in every turn of a loop, hidden from the compiler: it
// would make a copy of the loop for each value, and the instruction cache is short.
__device__ __forceinline__ bool opaque(bool b) {
  int v;
  asm volatile("mov.b32 %0, %1;" : "=r"(v) : "r"(static_cast<int>(b)));
  return v != 0;
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

// A warp's 32 rows of q, 8 elements of a row a lane: copied to where their halves will be,
// element 8 s of row r in chunk s % 8, swizzled by the row, of block s / 8.  Rows and
// columns that there are not become zeros.
template <int DP>
__device__ __forceinline__ uint32_t q_chunk(uint32_t q_at, int r, int sub) {
  return q_at + sub / 8 * (kRows * 128) + r * 128 + (((sub & 7) ^ (r & 7)) << 4);
}
template <bool F32Q, int DP>
__device__ __noinline__ void fetch_q(const AttnArgs &a, const Item &it, uint32_t q_at, int row0) {
  constexpr int TERMS = F32Q ? 2 : 1, SIZE = F32Q ? 4 : 2;
  constexpr int LR = DP / 8, RP = 32 / LR;    // lanes of a row, rows of a pass
  constexpr int kTerm = DP / 64 * kRows * 128;
  const int lane = threadIdx.x & 31, sub = lane % LR;
  const bool vec = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0 && a.ldq * SIZE % 16 == 0 &&
                   a.ldq_head * SIZE % 16 == 0;
  const int rows = it.rows, first = it.rt * kItemRows, head0 = it.h * a.G;
  const int64_t token0 = it.q.row0;
  // Row r of the lane's, its token and head; the next one is RP further.
  int r = lane / LR;
  const int rr = first + min(row0 + r, rows - 1);
  int tok = divide(rr, a.group), head = rr - tok * a.G;
  const uint8_t *token_at = static_cast<const uint8_t *>(a.q) +
                            ((token0 + tok) * a.ldq + head0 * a.ldq_head + 8 * sub) * SIZE;
#pragma unroll 1
  for (; r < 32; r += RP) {
    const bool on = row0 + r < rows && 8 * sub < a.cache.D;
    const uint8_t *from = on ? token_at + head * a.ldq_head * SIZE : static_cast<const uint8_t *>(a.q);
    head += RP;
    while (head >= a.G) {
      head -= a.G;
      token_at += a.ldq * SIZE;
    }
    const uint32_t dst = q_chunk<DP>(q_at, r, sub);
    if (opaque(vec) || !on) {
#pragma unroll
      for (int term = 0; term < TERMS; ++term)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + term * kTerm),
                     "l"(vec ? from + 16 * term : a.cache.k), "r"(on ? 16 : 0)
                     : "memory");
    } else {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        if (F32Q)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + (e >> 2) * kTerm + (e & 3) * 4),
                       "r"(reinterpret_cast<const uint32_t *>(from)[e])
                       : "memory");
        else
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + 2 * e),
                       "h"(reinterpret_cast<const uint16_t *>(from)[e])
                       : "memory");
      }
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Waits for the rows (a lane reads what it copied), scales them to halves, and notes what
// the scores are to be multiplied by.
template <bool F32Q, int DP>
__device__ __noinline__ void scale_q(const AttnArgs &a, uint32_t q_at, float *factors) {
  constexpr int TERMS = F32Q ? 2 : 1;
  constexpr int LR = DP / 8, RP = 32 / LR;
  constexpr int U = 2;
  constexpr int kTerm = DP / 64 * kRows * 128;
  const int lane = threadIdx.x & 31, sub = lane % LR;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
  for (int i = 0; i < 32 / RP; i += U) {
    // A few rows of a lane at a time, so that their steps overlap.
    uint32_t w[U][TERMS][4];
    float m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[u] = 0.0f;
#pragma unroll
      for (int term = 0; term < TERMS; ++term) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[u][term][0]), "=r"(w[u][term][1]), "=r"(w[u][term][2]),
                       "=r"(w[u][term][3])
                     : "r"(q_chunk<DP>(q_at, (i + u) * RP + lane / LR, sub) + term * kTerm)
                     : "memory");
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t b = w[u][term][e];
          if (F32Q)
            m[u] = fmaxf(m[u], fabsf(__uint_as_float(b)));
          else
            m[u] = max3(m[u], fabsf(__uint_as_float(b << 16)),
                        fabsf(__uint_as_float(b & 0xffff0000u)));
        }
      }
    }
#pragma unroll
    for (int o = LR / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = (i + u) * RP + lane / LR;
      const int e = min(max(8 - exponent_of(m[u]), -126), 126);
      const float up = power_of_two(e);
      uint32_t h[TERMS][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x, y;
        if (F32Q) {  // elements 2 k, 2 k + 1
          x = __uint_as_float(w[u][(TERMS - 1) * (k >> 1)][2 * (k & 1)]) * up;
          y = __uint_as_float(w[u][(TERMS - 1) * (k >> 1)][2 * (k & 1) + 1]) * up;
        } else {
          x = __uint_as_float(w[u][0][k] << 16) * up;
          y = __uint_as_float(w[u][0][k] & 0xffff0000u) * up;
        }
        h[0][k] = pack_half(x, y);
        if (TERMS == 2) {
          const float2 f = half2_floats(h[0][k]);
          h[TERMS - 1][k] = pack_half(x - f.x, y - f.y);
        }
      }
#pragma unroll
      for (int term = 0; term < TERMS; ++term)
        st_shared_v4(q_chunk<DP>(q_at, r, sub) + term * kTerm, h[term][0], h[term][1],
                     h[term][2], h[term][3]);
      if (sub == 0) factors[r] = power_of_two(-e) * a.scale_log2;
    }
  }
  __syncwarp();
}

// Where the scale of a tile's column lies: columns 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of 16 lie
// together, as a thread that makes weights has those.
__device__ __forceinline__ int scale_place(int col) {
  return (col & ~15) + ((col >> 1) & 3) * 4 + ((col >> 3) & 1) * 2 + (col & 1);
}

// Adds up beside the shares of the columns whose bits are set in `masks`, of a warp's rows,
// one a lane, which sees `limit` columns.  The scores are read again, from `scores` on,
// eight columns at a time: this is done before weights take their place.
__device__ __noinline__ void set_aside(uint32_t scores, uint32_t k_scales, const uint8_t *masks,
                                       int limit, float factor, float *far_top, float *far_sum) {
  float top = *far_top, sum = *far_sum;
#pragma unroll 1
  for (int j = 0; j < kTokens; j += 8) {
    const uint32_t mask = masks[j / 8];
    if (mask == 0) continue;
    float x[8], best = -INFINITY;
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]),
          "=f"(x[7])
        : "r"(scores + j)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float ks;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks) : "r"(k_scales + 4 * scale_place(j + i))
                   : "memory");
      x[i] = (mask >> i & 1) && j + i < limit ? x[i] * ks * factor : -INFINITY;
      best = fmaxf(best, x[i]);
    }
    const float from = best == -INFINITY ? 0.0f : best;
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) part += ex2(x[i] - from);
    add_share(top, sum, best, part);
  }
  *far_top = top;
  *far_sum = sum;
}

// A tile's scales of V where some lie far apart, or rows may be all zeros: log2 and
// reciprocal over the scales at `at`, 32 tokens apart, and the tile's head.  A row of zeros
// adds nothing to the result, whatever its scale: it must not take the others' weights
// towards a half's end, and so gets none.  Returns what the scales are relative to.
__device__ __noinline__ int rare_scales(const Cache &c, float *at, int *head, uint32_t firsts,
                                        uint32_t places, int e0, bool first) {
  const int lane = threadIdx.x & 31;
  uint32_t zeros = 0;
  int top = 0;         // positive numbers are in the order of their bits
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const float scale = at[32 * i];
    if (!(scale > 0.0f && scale < INFINITY)) continue;
    top = max(top, __float_as_int(scale));
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(firsts + 32 * 16 * i)
                 : "memory");
    uint32_t some = w[0] | w[1] | w[2] | w[3];
    int64_t place;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(place) : "r"(places + 32 * 8 * i) : "memory");
    const uint8_t *row = c.v + (place & ~1ll);
#pragma unroll 1
    for (int d = 16; d < c.D && (some & 0x7f7f7f7fu) == 0; d += 16) {
      const uint4 v = *reinterpret_cast<const uint4 *>(row + d);
      some |= v.x | v.y | v.z | v.w;
    }
    if ((some & 0x7f7f7f7fu) == 0) zeros |= 1u << i;
  }
  __syncwarp();
  top = min(exponent_of(__int_as_float(__reduce_max_sync(0xffffffffu, top))), 126);
  const int rise = top > e0 + kSpan ? top - e0 : 0;
  e0 += rise;
  uint32_t any = 0;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const float scale = at[32 * i], v = scale * power_of_two(-e0);
    const bool fine = scale > 0.0f && scale < INFINITY, zero = zeros >> i & 1;
    const bool less = fine && (zero || exponent_of(scale) < e0 - kSpan);
    const uint32_t far = __ballot_sync(0xffffffffu, less);
    any |= far;
    at[32 * i] = !fine ? NAN : !less ? lg2(v) : zero ? -INFINITY : log2_far(scale, e0);
    at[32 * i + kTokens] = !fine ? 1.0f : less ? 0.0f : rcp(v);
    if (lane == 0) head[4 + i] = static_cast<int>(far);
  }
  if (lane == 0) {
    head[0] = e0;
    head[1] = (rise > 0 && !first ? 1 : 0) | (any ? 2 : 0);
    head[2] = rise;
  }
  return e0;
}

// Columns k .. k+15 of V that hold a code that is not finite at a token that a row sees,
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
    for (int i = 0; i < 16; ++i)
      if (!Fm::finite(codes[k + i])) bad |= 1u << i;
  }
  return bad;
}

// Joins a row's sums with what the pieces of its part before this one made, over them in
// tensor memory, a row a lane.
__device__ __noinline__ Total join_pieces(uint32_t o_tm, const float *before, const float *lse,
                                          int D, bool on, Total t) {
  const Weights w = on ? weigh(t.lse, *lse) : Weights{1.0f, 0.0f, t.lse, 1.0f};
#pragma unroll 1
  for (int k = 0; k < D; k += 16) {
    float o[16];
    __syncwarp();
    tmem_load16(o_tm + k, o);
    if (on) {
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = joined(w, o[i] * t.f0 * t.f1, before[k + i]);
    }
    __syncwarp();
    tmem_store16(o_tm + k, o);
  }
  tmem_wait_store();
  return {w.lse, 1.0f, 1.0f};
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
  // The same in all lanes, which the compiler would not see otherwise.
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t bars = base + C::kBar;
  auto full_bar = [&](int i) { return bars + 8u * i; };                       // K or V
  auto empty_bar = [&](int i) { return bars + 8u * (C::SLOTS + i); };
  auto scfull_bar = [&](int i) { return bars + 8u * (2 * C::SLOTS + i); };    // scales
  auto scfree_bar = [&](int i) { return bars + 8u * (2 * C::SLOTS + kScaleBufs + i); };
  auto atfull_bar = [&](int i) { return bars + 8u * (2 * C::SLOTS + 2 * kScaleBufs + i); };
  auto atfree_bar = [&](int i) { return bars + 8u * (2 * C::SLOTS + 3 * kScaleBufs + i); };
  const uint32_t rest = bars + 8u * (2 * C::SLOTS + 4 * kScaleBufs);
  // Of tile t of rows: its scores, the weights of half h of the tokens, the first half's
  // products in O, an item's O, and that it has been read.
  auto s_bar = [&](int t) { return rest + 8u * t; };
  auto p_bar = [&](int t, int h) { return rest + 8u * (2 + 2 * t + h); };
  auto pv_bar = [&](int t) { return rest + 8u * (6 + t); };
  auto o_bar = [&](int t) { return rest + 8u * (8 + t); };
  auto ofree_bar = [&](int t) { return rest + 8u * (10 + t); };
  const uint32_t qfull_bar = rest + 8u * 12, done_bar = rest + 8u * 13;
  auto itfull_bar = [&](int i) { return rest + 8u * (14 + i); };
  auto itfree_bar = [&](int i) { return rest + 8u * (14 + kItemBufs + i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sbase + C::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + C::kMisc + 4);
  volatile int *poison = reinterpret_cast<volatile int *>(sbase + C::kMisc + 8);
  float *factors = reinterpret_cast<float *>(sbase + C::kFactors);
  __shared__ volatile int more_tiles[kScaleBufs];
  __shared__ Item items[kItemBufs];
  __shared__ Walk walk;
  __shared__ int page_ids[2][kTokens];
  __shared__ float row_stats[8][64];
  // Of a warp's rows: the maximum and the sum of add_share; what V's scales are relative to.
  __shared__ float beside[8][65];
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(full_bar(i), kTokens / kGroup);
      mbar_init(empty_bar(i), 1);
    }
    for (int i = 0; i < kScaleBufs; ++i) {
      mbar_init(atfull_bar(i), 1);
      mbar_init(atfree_bar(i), kConverters);
      mbar_init(scfull_bar(i), 2);
      mbar_init(scfree_bar(i), 8);
    }
    for (int i = 0; i < kItemBufs; ++i) {
      mbar_init(itfull_bar(i), 1);
      mbar_init(itfree_bar(i), kItemReaders);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_bar(t), 1);
      mbar_init(p_bar(t, 0), 4);
      mbar_init(p_bar(t, 1), 4);
      mbar_init(pv_bar(t), 1);
      mbar_init(o_bar(t), 1);
      mbar_init(ofree_bar(t), 4);
    }
    mbar_init(qfull_bar, 8);
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    *poison = 0;
    fence_mbar_init();
  }
  if (warp == 15) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) a.desc[blockIdx.x].parts = 0;
  share_out<kThreads, kItemRows, kTokens, kItemCost>(a, &sh, warp_sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
           wait_long(bar, parity, timeout_ns, a.rows.status, abort_flag);
  };
  // Items come from warp 13 through a ring; every warp that wants them takes each in
  // turn: number n, or none where the work is done.
  auto item_ready = [&](uint32_t n, bool &ok) {
    ok = wait(itfull_bar(n % kItemBufs), (n / kItemBufs) & 1u);
    return ok && items[n % kItemBufs].count > 0;
  };
  auto item_done = [&](uint32_t n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(itfree_bar(n % kItemBufs));
  };

  if (warp < 8) {
    // --------------------------------------------------- scores to weights
    // A thread holds the columns 8 i + 2 c + {0, 1} of four rows, g + 8 u of its warp's
    // 32, as a thread of one row would have to read every column's scales.
    const int t = warp >> 2;                    // tile
    const int row0 = t * kRows + (warp & 3) * 32, g = lane >> 2, c = lane & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_tm = lanes + C::kS + 128 * t, o_tm = lanes + C::kO + DP * t;
    constexpr uint32_t kLanes16 = 16u << 16;
    uint32_t sc = 0;      // tiles of tokens so far
    uint32_t tiles = 0;   // those of them that this tile of rows took part in
    uint32_t o_uses = 0;  // items that it took part in
    const uint32_t q_at = base + t * TERMS * C::kTileBytes + (warp & 3) * 32 * 128;
    float *const my_factors = factors + row0;
    auto q_done = [&] {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull_bar);
    };
    bool ok, more = item_ready(0, ok);
    if (more) {
      fetch_q<F32Q, DP>(a, items[0], q_at, row0);
      scale_q<F32Q, DP>(a, q_at, my_factors);
      q_done();
    }
    for (uint32_t n = 0; ok && more; ++n) {
      const Item &it = items[n % kItemBufs], &upcoming = items[(n + 1) % kItemBufs];
      const int rows = it.rows, count = it.count, tok0 = it.tile0 * kTokens;
      const bool active = t * kRows < rows;
      float factor[4], M[4];
      uint64_t l2[4];                  // of even and odd columns
      float *const far_top = beside[warp], *const far_sum = beside[warp] + 32;
      far_top[lane] = -INFINITY;
      far_sum[lane] = 0.0f;
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        factor[u] = my_factors[8 * u + g];
        M[u] = -INFINITY;
        l2[u] = pair(0.0f, 0.0f);
      }
      // Tokens that each row of the warp sees: the first one's.
      const int all = row0 + 32 <= rows ? tokens_seen(a, it.q, it.rt * kItemRows + row0) : 0;
#pragma unroll 1
      for (int j = 0; j < count; ++j, ++sc) {
        const int buf = sc % kScaleBufs;
        if (!(ok = wait(scfull_bar(buf), (sc / kScaleBufs) & 1u))) break;
        if (j + 1 == count) {
          more = item_ready(n + 1, ok);
          if (!ok) break;
        }
        if (!opaque(active)) {
          if (lane == 0) mbar_arrive(scfree_bar(buf));
          continue;
        }
        const uint32_t scales = base + C::kScales + buf * kScaleBytes;
        const int *const head = reinterpret_cast<const int *>(
            sbase + C::kScales + buf * kScaleBytes + kTileHead);
        if (j == 0) far_top[64] = __int_as_float(head[0]);
        const int apart = head[1];
        if (!(ok = wait(s_bar(t), tiles & 1u))) break;
        tc_fence_after();
        if (opaque(apart)) {
          if (apart & 1) {
            const int rise = head[2];
            far_top[64] = __int_as_float(head[0]);
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
              float y, z;
              const uint64_t l = u < 2 ? (u == 0 ? l2[0] : l2[1]) : (u == 2 ? l2[2] : l2[3]);
              const float m = u < 2 ? (u == 0 ? M[0] : M[1]) : (u == 2 ? M[2] : M[3]);
              unpair(l, y, z);
              y += z;
              y += __shfl_xor_sync(0xffffffffu, y, 1);
              y += __shfl_xor_sync(0xffffffffu, y, 2);
              if (c == 0) add_share(far_top[8 * u + g], far_sum[8 * u + g], m - kShift, y);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              M[u] -= static_cast<float>(rise);
              l2[u] = pair(0.0f, 0.0f);
            }
            __syncwarp();
          }
          if (apart & 2) {
            const int r = row0 + lane;
            const int seen = r < rows ? tokens_seen(a, it.q, it.rt * kItemRows + r) : 0;
            set_aside(s_tm, scales, reinterpret_cast<const uint8_t *>(head + 4),
                      seen - tok0 - j * kTokens, my_factors[lane], far_top + lane, far_sum + lane);
            __syncwarp();
          }
        }
        // The last scores of these rows are made: the next rows may take their place.
        if (j + 1 == count && more) fetch_q<F32Q, DP>(a, upcoming, q_at, row0);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          constexpr int HT = kTokens / 2;
          const uint32_t hs = scales + 4 * HT * half + 16 * c;
          float x[2][32];
#pragma unroll
          for (int b = 0; b < 2; ++b) tmem_load_rows(s_tm + HT * half + b * kLanes16, x[b]);
          tmem_wait32(x[0]);
          tmem_wait32(x[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint64_t ks[2], lv[2];
            lds_pairs(hs + 64 * i, ks[0], ks[1]);
            lds_pairs(hs + 4 * kTokens + 64 * i, lv[0], lv[1]);
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                float *v = &x[u >> 1][4 * (2 * i + p) + 2 * (u & 1)];
                unpair(fma2(mul2(pair(v[0], v[1]), ks[p]), pair(factor[u], factor[u]), lv[p]),
                       v[0], v[1]);
              }
          }
          const int first = tok0 + j * kTokens + HT * half;
          if (first + HT > all) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int r = row0 + 8 * u + g;
              const int seen = r < rows ? tokens_seen(a, it.q, it.rt * kItemRows + r) : 0;
              const int limit = seen - first - 2 * c;
#pragma unroll
              for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (8 * i + e >= limit) x[u >> 1][4 * i + 2 * (u & 1) + e] = -INFINITY;
            }
          }
          float best[4];
          bool raise = false;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float *v = &x[u >> 1][2 * (u & 1)];
            best[u] = fmaxf(v[0], v[1]);
#pragma unroll
            for (int i = 1; i < 8; ++i) best[u] = max3(best[u], v[4 * i], v[4 * i + 1]);
            raise |= best[u] > M[u] + kLazy;
          }
          if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              float m = fmaxf(best[u], M[u]);
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
              best[u] = m == -INFINITY ? 1.0f : ex2(M[u] - m);
              M[u] = m;
              l2[u] = mul2(l2[u], pair(best[u], best[u]));
            }
            if (j + half > 0) {
              // The products of the tile before are in O, as the scores came after them.
              if (half > 0 && !(ok = wait(pv_bar(t), tiles & 1u))) break;
              tc_fence_after();
#pragma unroll 1
              for (int k = 0; k < DP / 16; ++k) {
                // 16 lanes of 32 columns at a time.
                const uint32_t at = o_tm + (k >> 1) * 32 + (k & 1) * kLanes16;
                const float d0 = k & 1 ? best[2] : best[0], d1 = k & 1 ? best[3] : best[1];
                float o[16];
                tmem_load_rows16(at, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= i & 2 ? d1 : d0;
                tmem_store_rows16(at, o);
              }
            }
          }
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint64_t top[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float v = M[2 * b + u] == -INFINITY ? 0.0f : kShift - M[2 * b + u];
              top[u] = pair(v, v);
            }
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint64_t iv[2];
              lds_pairs(hs + 8 * kTokens + 64 * i, iv[0], iv[1]);
#pragma unroll
              for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const float *v = &x[b][4 * (2 * i + p) + 2 * u];
                  float y, z;
                  unpair(add2(pair(v[0], v[1]), top[u]), y, z);
                  y = ex2(y);
                  z = ex2(z);
                  l2[2 * b + u] = fma2(pair(y, z), iv[p], l2[2 * b + u]);
                  w[2 * (2 * i + p) + u] = pack_half(y, z);
                }
            }
            tmem_store_halves(s_tm + HT / 2 * half + b * kLanes16, w);
          }
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
      if (more) {
        if (!active) {
          // These warps wait for no scores: without this one that is tiles ahead of the
          // other row tile's would arrive for item n + 1 in item n's place.
          if (!(ok = wait(qfull_bar, n & 1u))) break;
          fetch_q<F32Q, DP>(a, upcoming, q_at, row0);
        }
        scale_q<F32Q, DP>(a, q_at, my_factors);
        q_done();
      }
      if (!active) {
        item_done(n);
        continue;
      }
      // A row to each lane from here on.
      float sum, best;
      {
        float *stats = row_stats[warp];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float y, z;
          unpair(l2[u], y, z);
          y += z;
          y += __shfl_xor_sync(0xffffffffu, y, 1);
          y += __shfl_xor_sync(0xffffffffu, y, 2);
          if (c == 0) {
            stats[8 * u + g] = y;
            stats[32 + 8 * u + g] = M[u];
          }
        }
        __syncwarp();
        sum = stats[lane];
        best = stats[32 + lane];
      }
      const int row = (warp & 3) * 32 + lane;     // of the tile
      const int r = it.rt * kItemRows + min(row0 + lane, rows - 1);
      const int my_seen = row0 + lane < rows ? tokens_seen(a, it.q, r) : 0;
      // The rows' results.
      if (!(ok = wait(o_bar(t), o_uses & 1u))) break;
      ++o_uses;
      tc_fence_after();
      Total all_of = total_of(best - kShift, sum, far_top[lane], far_sum[lane],
                                    __float_as_int(far_top[64]));
      const bool mask = *poison != 0;
      const bool on = row0 + lane < rows;
      const bool whole = it.first == 0 && it.tile0 + it.count == it.tiles;
      const int tok = divide(r, a.group);
      const int64_t out_row = static_cast<int64_t>(it.q.row0) + tok;
      const int hq = it.h * a.G + r - tok * a.G;
      const int64_t place = out_row * a.Hq + hq;
      const int64_t part =
          (2 * static_cast<int64_t>(blockIdx.x) + (it.first > 0 ? 0 : 1)) * kItemRows + t * kRows + row;
      if (opaque(it.after))
        all_of = join_pieces(o_tm, a.part_o + part * DP, a.part_lse + part, a.cache.D, on, all_of);
      const float lse = all_of.lse;
      Weights weights = {1.0f, 0.0f, lse, 1.0f};
      const float *pre = nullptr;
      if (whole && !a.raw_o && on) {
        weights = weigh(a, out_row, hq, lse);
        if (a.pre_o) pre = a.pre_o + place * a.cache.D;
        if (a.lse) a.lse[out_row * a.ld_lse + hq] = weights.lse * kLn2;
      } else if (on) {
        (whole ? a.raw_lse + place : a.part_lse + part)[0] = lse;
      }
      float *const f32 = !whole ? a.part_o + part * DP
                         : a.raw_o ? a.raw_o + place * a.cache.D : nullptr;
      uint16_t *const b16 = a.out + out_row * a.ldo + hq * a.ldo_head;
      const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | a.ldo * 2 | a.ldo_head * 2) & 31) == 0;
#pragma unroll 1
      for (int k = 0; k < a.cache.D; k += 16) {
        float o[16];
        tmem_load16(o_tm + k, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = o[i] * all_of.f0 * all_of.f1;
        if (opaque(mask && on)) {
          const uint32_t bad = lost_columns<Fm>(a, it, my_seen, k);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (bad >> i & 1u) o[i] = NAN;
        }
        if (!opaque(on)) continue;
        if (opaque(f32 != nullptr)) {
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(o[i + e]);
            store32(f32 + k + i, u);
          }
          continue;
        }
        if (opaque(pre != nullptr)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = joined(weights, o[i], pre[k + i]);
        }
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
          u[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        if (opaque(wide)) {
          store32(b16 + k, u);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) b16[k + i] = static_cast<uint16_t>(u[i / 2] >> (16 * (i & 1)));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree_bar(t));
      if (threadIdx.x == 0 && !whole && !it.more && it.first == 0)
        a.desc[blockIdx.x] = {it.s, it.h, it.rt,
                              owner_of(sh, it.end - 1) - static_cast<int>(blockIdx.x) + 1};
      item_done(n);
    }
  } else if (warp < 8 + kConverters) {
    // ------------------------------------------------- codes to halves
    // Jobs n = w, w + 5, ...: job n is group n % 8 of K (n % 16 < 8) or V of tile n / 16.
    // A lane reads back what it copied itself.
    constexpr int CH = DP / 16;        // 16-byte chunks of a row
    constexpr int PER = CH / 2;        // of a lane in a job
    const uint32_t raw = base + C::kRaw + (warp - 8) * (C::AHEAD * C::kJob) + lane * 16;
    // The lane's chunk i.  Eight lanes cover even chunks of halves that are swizzled by
    // the token, so two tokens, one of them odd.
    const int ch = DP == 128 ? lane & 7 : lane & 3;
    const int tok = DP == 128 ? (lane >> 3) * 2 + ((lane >> 2) & 1) : lane >> 2;
    auto local = [&](int i) { return DP == 128 ? (i >> 1) * 8 + (tok ^ (i & 1)) : i * 8 + tok; };
    uint32_t jobs = 0xffffffffu;       // until the last tile's places say so
    uint32_t flags = 0;                // of the jobs under way: not all rows see the tile
    bool ok = true;
    auto request = [&](uint32_t n) {
      bool partial = false;
      if (n < jobs) {
        const uint32_t tile = n / kJobs, buf = tile % kScaleBufs;
        if (!(ok = wait(atfull_bar(buf), (tile / kScaleBufs) & 1u))) return;
        if (!more_tiles[buf]) jobs = tile * kJobs;
        if (n >= jobs) return;
        const bool is_v = n & (kJobs / 2);
        const uint8_t *codes = is_v ? a.cache.v : a.cache.k;
        const uint32_t from = base + C::kPlaces + (buf * kTokens + n % (kJobs / 2) * kGroup) * 8;
        const uint32_t dst = raw + n / kConverters % C::AHEAD * C::kJob;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          int64_t o;
          asm volatile("ld.shared.b64 %0, [%1];" : "=l"(o) : "r"(from + local(i) * 8) : "memory");
          // The lowest bit of a place marks a tile that not all rows see.
          partial = is_v && (o & 1);
          const bool on = o >= 0 && ch * 16 < a.cache.D;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * 512),
                       "l"(codes + (on ? (o & ~1ll) + ch * 16 : 0)), "r"(on ? 16 : 0)
                       : "memory");
        }
        if ((n + kConverters) / kJobs != tile) {  // the last of this tile's
          __syncwarp();
          if (lane == 0) mbar_arrive(atfree_bar(buf));
        }
      }
      flags |= (partial ? 1u : 0u) << (C::AHEAD - 1);
    };
#pragma unroll 1
    for (uint32_t n = warp - 8; ok; n += kConverters) {
      // The first rounds only request.
      if (n >= C::AHEAD * kConverters) {
        const uint32_t m = n - C::AHEAD * kConverters;
        if (m >= jobs) break;
        const uint32_t use = m / (kJobs / 2), slot = use % C::SLOTS;
        if (!(ok = wait(empty_bar(slot), ((use / C::SLOTS) & 1u) ^ 1u))) break;
        asm volatile("cp.async.wait_group %0;" ::"n"(C::AHEAD - 1) : "memory");
        const uint32_t src = raw + m / kConverters % C::AHEAD * C::kJob;
        const uint32_t dst = base + C::kRing + slot * C::kTileBytes + (ch >> 2) * C::kBlock +
                             m % (kJobs / 2) * (kGroup * 128);
        bool found = false;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          uint32_t w[4], h[8];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(src + i * 512)
                       : "memory");
          if (opaque(flags & 1u)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) found |= Fm::clear4(w[q]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            h[2 * q] = decode2<FMT>(w[q] & 0xffffu);
            h[2 * q + 1] = decode2<FMT>(w[q] >> 16);
          }
          const uint32_t r = local(i), row = dst + r * 128;
          const uint32_t c0 = 2 * (ch & 3), sw = r & 7;
          st_shared_v4(row + ((c0 ^ sw) << 4), h[0], h[1], h[2], h[3]);
          st_shared_v4(row + (((c0 + 1) ^ sw) << 4), h[4], h[5], h[6], h[7]);
        }
        if (found) *poison = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full_bar(slot));
      }
      flags >>= 1;
      request(n);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp < 15) {
    // ------------------------------------------------- places and scales
    // A lane has four tokens of a tile, 32 apart.  In turn `step`, page numbers of tile
    // step + 1 and scales of tile step are requested, by copies into shared memory, and
    // the scales of tile step - 1 are written.
    const bool is_v = warp == 14;
    const Cache &c = a.cache;
    const float *const scales_from = is_v ? c.v_scale : c.k_scale;
    const int scale_at = scale_place(lane);
    const uint32_t page16 = static_cast<uint32_t>(c.page_stride >> 4),
                   token16 = static_cast<uint32_t>(c.token_stride >> 4),
                   head16 = static_cast<uint32_t>(c.head_stride >> 4);
    const uint32_t s_page = static_cast<uint32_t>(c.scale_page_stride),
                   s_token = static_cast<uint32_t>(c.scale_token_stride),
                   s_head = static_cast<uint32_t>(c.scale_head_stride);
    const uint32_t pages = smem_addr(page_ids[warp - 13]) + 4 * lane;
    auto scales_of = [&](int step) {
      return base + C::kScales + step % kScaleBufs * kScaleBytes;
    };
    auto copy4 = [&](uint32_t dst, const void *src) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
    };
    int pj = 0, h = 0, e0 = 0, tok0 = 0, most = 0;
    uint32_t n_item = 0;
    bool partial = false, first = false, was_first = false, have = false, ok = true;
    if (!is_v && lane == 0) start_walk<kItemRows>(a, sh, &walk);
    // The first turn only requests page numbers.
#pragma unroll 1
    for (int step = -1; ok; ++step) {
      const bool here = have;
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (here) {
        const int buf = step % kScaleBufs;
        ok = wait(scfree_bar(buf), ((step / kScaleBufs) & 1u) ^ 1u);
        if (ok && !opaque(is_v)) ok = wait(atfree_bar(buf), ((step / kScaleBufs) & 1u) ^ 1u);
        if (!ok) break;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int tk = tok0 + lane + 32 * i;
          int p;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(p) : "r"(pages + 128 * i) : "memory");
          const bool in = tk < most, good = in && p >= 0 && p < c.num_pages;
          if (in && !good) atomicOr(a.rows.status, kStatusBadDeviceArg);
          const uint64_t pl = tk - divide(tk, c.page) * c.page_size;
          const uint32_t dst = scales_of(step) + 4 * (scale_at + 32 * i + (opaque(is_v) ? kTokens : 0));
          if (opaque(is_v)) {
            const uint64_t at = (static_cast<uint64_t>(p) * page16 + pl * token16 +
                                 static_cast<uint64_t>(h) * head16) * 16;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             base + C::kFirst + ((step & 1) * kTokens + lane + 32 * i) * 16),
                         "l"(c.v + (good ? at : 0)), "r"(good ? 16 : 0)
                         : "memory");
          }
          if (good)
            copy4(dst, scales_from + static_cast<uint64_t>(p) * s_page + pl * s_token +
                           static_cast<uint64_t>(h) * s_head);
          else
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst),
                         "f"(in ? NAN : is_v ? 0.0f : 1.0f) : "memory");
          if (!opaque(is_v)) {
            // Lowest bit: not all rows see the tile.  All bits: there is no token.
            const uint64_t at = good ? (static_cast<uint64_t>(p) * page16 + pl * token16 +
                                        static_cast<uint64_t>(h) * head16) * 16 + (partial ? 1 : 0)
                                     : ~0ull;
            asm volatile("st.shared.b64 [%0], %1;" ::"r"(
                             base + C::kPlaces + (buf * kTokens + lane + 32 * i) * 8),
                         "l"(at)
                         : "memory");
          }
        }
      }
      const bool now_first = first;
      // The next tile, of this item or the next, which warp 13 makes.
      if (step < 0 || (here && pj == items[n_item % kItemBufs].count)) {
        pj = 0;
        if (step >= 0) {
          if (opaque(is_v)) item_done(n_item);
          ++n_item;
        }
        const int i = n_item % kItemBufs;
        ok = wait(opaque(is_v) ? itfull_bar(i) : itfree_bar(i),
                  ((n_item / kItemBufs) & 1u) ^ (opaque(is_v) ? 0u : 1u));
        if (!ok) break;
        if (!opaque(is_v)) {
          if (lane == 0) {
            if (!next_item<kItemRows, kTokens, kItemCost, kPiece>(a, &walk, &items[i])) items[i].count = 0;
            mbar_arrive(itfull_bar(i));
          }
          __syncwarp();
        }
        have = items[i].count > 0;
      }
      if (have) {
        const Item &it = items[n_item % kItemBufs];
        const int all = tokens_seen(a, it.q, it.rt * kItemRows);
        most = tokens_seen(a, it.q, it.rt * kItemRows + it.rows - 1);
        const int32_t *table = a.rows.table + it.s * a.rows.ld_table;
        tok0 = (it.tile0 + pj) * kTokens;
        h = it.h;
        first = pj == 0;
        partial = tok0 + kTokens > all && all < most;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int tk = tok0 + lane + 32 * i;
          if (tk < most) copy4(pages + 128 * i, table + divide(tk, c.page));
        }
        ++pj;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (step < 0) continue;
      if (!opaque(is_v)) {
        const int buf = step % kScaleBufs;
        if (!here && !(ok = wait(atfree_bar(buf), ((step / kScaleBufs) & 1u) ^ 1u))) break;
        if (lane == 0) more_tiles[buf] = here;
        __syncwarp();
        if (lane == 0) mbar_arrive(atfull_bar(buf));
      }
      if (step > 0) {
        // Of the tile before, whose scales have come.
        float *out = reinterpret_cast<float *>(smem_raw + (scales_of(step - 1) - raw));
        __syncwarp();
        if (opaque(is_v)) {
          // Relative to a power of two near the scale of the item's first token.
          if (was_first) e0 = min(exponent_of(out[kTokens]), 126);
          // Whether the exponents (of subnormal numbers one less than exponent_of) are within
          // e0 - kSpan .. e0 + kSpan, and whether rows of V may be all zeros: nearly all have
          // another code among the first 16.
          const uint32_t low = static_cast<uint32_t>(e0 + 127 - kSpan);
          const float down = power_of_two(-e0);
          const uint32_t firsts = base + C::kFirst + (((step - 1) & 1) * kTokens + lane) * 16;
          bool rare = false;
          float scale[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(firsts + 32 * 16 * i)
                         : "memory");
            scale[i] = out[kTokens + 32 * i + scale_at];
            const bool fine = scale[i] > 0.0f && scale[i] < INFINITY;
            rare |= fine && ((__float_as_uint(scale[i]) >> 23) - low > 2 * kSpan ||
                             ((w[0] | w[1] | w[2] | w[3]) & 0x7f7f7f7fu) == 0);
          }
          int *const head = reinterpret_cast<int *>(out) + kTileHead / 4;
          if (__any_sync(0xffffffffu, rare)) {
            const int buf = (step - 1) % kScaleBufs;
            if (!(ok = wait(atfull_bar(buf), ((step - 1) / kScaleBufs) & 1u))) break;
            e0 = rare_scales(a.cache, out + kTokens + scale_at, head, firsts,
                             base + C::kPlaces + (buf * kTokens + lane) * 8, e0, was_first);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float *at = out + kTokens + 32 * i + scale_at;
              const float v = scale[i] * down;
              const bool fine = scale[i] > 0.0f && scale[i] < INFINITY;
              float lg, inv;
              asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(v));
              asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(v));
              at[0] = fine ? lg : NAN;
              // A bad scale is in the exponent alone: rows that do not see it have weight 0.
              at[kTokens] = fine ? inv : 1.0f;
            }
            if (lane == 0) {
              head[0] = e0;
              head[1] = 0;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(scfull_bar((step - 1) % kScaleBufs));
      }
      if (!here) break;
      was_first = now_first;
    }
  } else {
    {
      // ----------------------------------------------------------- MMAs
      constexpr int HT = kTokens / 2;
      constexpr uint32_t s_idesc = idesc_f16(kTokens, false), o_idesc = idesc_f16(DP, true);
      const uint64_t q_desc = smem_desc_k128_sw128(base);
      const uint64_t k_desc = smem_desc_k128_sw128(base + C::kRing);
      const uint64_t v_desc = smem_desc_mn_sw128(base + C::kRing, C::kBlock);
      uint32_t s_step = 0, v_step = 0;      // tiles of tokens of S and of O
      uint32_t p_uses[2] = {0, 0}, o_uses[2] = {0, 0};
      // S of tile t against the K tile s_step.
      auto scores = [&](int t) {
        const uint64_t ad = q_desc + t * (TERMS * C::kTileBytes / 16);
        const uint64_t bd = k_desc + (2 * s_step) % C::SLOTS * (C::kTileBytes / 16);
        const uint32_t d = tmem + C::kS + 128 * t;
#pragma unroll
        for (int term = 0; term < TERMS; ++term)
#pragma unroll
          for (int b = 0; b < DP / 64; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              umma_ss(d, ad + (term * C::kTileBytes + b * C::kBlock) / 16 + 2 * q,
                      bd + b * C::kBlock / 16 + 2 * q, s_idesc, term > 0 || b > 0 || q > 0);
        commit(s_bar(t));
      };
      auto k_ready = [&] {
        const bool r = wait(full_bar((2 * s_step) % C::SLOTS), ((2 * s_step) / C::SLOTS) & 1u);
        tc_fence_after();
        return r;
      };
      auto k_done = [&] {
        commit(empty_bar((2 * s_step) % C::SLOTS));
        ++s_step;
      };
      bool ok;
      for (uint32_t n = 0; item_ready(n, ok); ++n) {
        // An item's first scores come after all of the last one's products, which the
        // warps that bring its rows may wait for.
        const int rows = items[n % kItemBufs].rows, count = items[n % kItemBufs].count;
        item_done(n);
        // Turn j: the products of tile j, then the scores of tile j + 1 of the item; an
        // item's first scores come after all of the last one's products, which the warps
        // that bring its rows may wait for.
#pragma unroll 1
        for (int j = -1; ok && j < count; ++j) {
          const bool last = j + 1 == count;
          const int v_slot = (2 * v_step + 1) % C::SLOTS;
          if (j >= 0) ok = wait(full_bar(v_slot), ((2 * v_step + 1) / C::SLOTS) & 1u);
#pragma unroll 1
          for (int t = 0; ok && t * kRows < rows; ++t) {
            if (j >= 0) {
#pragma unroll 1
              for (int half = 0; half < 2; ++half) {
                ok = wait(p_bar(t, half), (t ? p_uses[1] : p_uses[0]) & 1u);
                if (ok && j + half == 0 && (t ? o_uses[1] : o_uses[0]) > 0)
                  ok = wait(ofree_bar(t), ((t ? o_uses[1] : o_uses[0]) - 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                const uint64_t bd = v_desc + (v_slot * C::kTileBytes + half * (HT * 128)) / 16;
                const uint32_t d = tmem + C::kO + DP * t, p = tmem + C::kS + 128 * t + HT / 2 * half;
#pragma unroll
                for (int q = 0; q < HT / 16; ++q)
                  umma_ts(d, p + 8 * q, bd + q * (2048 / 16), o_idesc, j + half > 0 || q > 0);
                if (half == 0) commit(pv_bar(t));
              }
              if (!ok) break;
              ++(t ? p_uses[1] : p_uses[0]);
              if (j == 0) ++(t ? o_uses[1] : o_uses[0]);
              if (last) commit(o_bar(t));
            }
            if (!last) {
              if (t == 0) {
                ok = (j >= 0 || wait(qfull_bar, n & 1u)) && k_ready();
                if (!ok) break;
              }
              scores(t);
            }
          }
          if (!ok) break;
          if (j >= 0) {
            commit(empty_bar(v_slot));
            ++v_step;
          }
          if (!last) k_done();
        }
        if (!ok) break;
      }
      commit(done_bar);
      mbar_wait_drain(done_bar, 0, timeout_ns, a.rows.status);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 15) {
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

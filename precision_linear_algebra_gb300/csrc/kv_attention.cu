// Attention of few rows of each sequence over the FP8 key/value cache, the join
// of partial results, and the entry point.
//
// A row (token t, query head h) of sequence s has scores x_j = (q . k_j) ks_j
// scale over the tokens j that it sees, k_j the codes of K's row and ks_j its
// scale; out = sum_j p_j vs_j v_j / sum_j p_j, p_j = exp(x_j).  V's scales go into
// the exponent, w_j = 2^(x_j log2 e + log2 vs_j - M) with a running maximum M of
// those sums, so that the products are w_j times codes, and the denominator is
// sum_j w_j / vs_j.  One exponential an element, no product with dequantised values.
// Where V's scales lie far apart, the denominator has a second part (kSpan), and so it has
// for rows of zeros in V, which would otherwise set M by a scale that scales nothing.
//
// Precision: codes are halves exactly.  A BF16 query row, scaled by a power of
// two to a maximum of 2^8, is halves exactly but for elements below 2^-22 of its
// maximum (off by 2^-33 of it at most); an FP32 one is the sum of two halves,
// 2^-22.  w_j is rounded to a half, 2^-11, at most 2^7 (2^15 between two rescalings),
// so that only what is 2^-21 of the largest or less loses more; unrounded in the
// denominator.  Halves because the result is BF16 and mma.sync has no wider type that the
// codes fit without a loss of rate.  Sums are FP32, in pieces (kPiece).
//
// Bound: HBM, K's and V's codes once for all heads of a group.  A warp streams 32
// tokens at a time through a ring of its own, two steps deep, filled by TMA (16 tokens
// of a page a copy) or, where pages are not made of whole groups of 16, by cp.async in
// chunks of 16 bytes: no barrier in the loop.  mma.sync m16n8k16 takes 16 rows, which is
// what a group of heads of one token needs; the fragments come from codes by one
// conversion for two of them.  tcgen05 wants 64 rows at least, which kv_attention_tc.cu
// has.  Measured, 8 K/V heads of 128 with 8 query heads each, the join included: 64
// sequences of 8192 tokens 181 us (6.1 TB/s), of lengths up to 8192 108 us (5.6; 128 with
// steps of 32 tokens, 149 with 16, both before kItemCost); one of 131072 60 us (4.7); one
// of 2048 17 us, two launches whose addresses and instructions come one after the other;
// 256 of 1024 115 us (4.9).  Items of few tiles are bound by the fetching of instructions:
// what they seldom need (shares beside, codes that are not finite, the ends of pages) is
// kept out of their way, in loops of its own and out of line.
#include "kv_attention.cuh"

namespace fp8la {
namespace kv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kRows = kFewItemRows;  // rows of a tile
constexpr int kGroup = 16;      // tokens that TMA brings at once
constexpr int kSubs = 2;        // groups of a warp's step
constexpr int kStep = kSubs * kGroup;
constexpr int kTile = kWarps * kStep;
static_assert(kTile == kTileTokens, "what the prefix's units are counted in");
// What an item costs beside its tiles, in tiles.  64 requests of up to 8192 tokens, us,
// with 0 to 5: 141, 130, 121, 110, 109, 110.
constexpr int kItemCost = kFewItemCost;
constexpr int kStages = 2;
constexpr float kShift = 7.0f;  // w of the running maximum is 2^7
constexpr float kLazy = 8.0f;   // it is raised where 2^8 is passed

template <bool F32Q, int DP>
struct Cfg {
  static constexpr int CH = DP / 16;                  // 16-byte chunks of a row
  static constexpr int kK = kGroup * DP;
  static constexpr int kStage = kSubs * 2 * kK;       // of a warp: K and V of each group
  static constexpr int kRing = kStages * kStage;
  static constexpr int kScales = kWarps * kRing;      // ks, log2 vs, 1 / vs of each stage
  static constexpr int kScaleStage = 3 * kStep * 4;
  static constexpr int kBar = kScales + kWarps * kStages * kScaleStage;
  static constexpr int KS = DP / 16;                  // MMA steps along D
  static constexpr int TERMS = F32Q ? 2 : 1;
  static constexpr bool QREG = KS * TERMS <= 8;
  static constexpr int kQ = kBar + kWarps * kStages * 8;  // query fragments
  static constexpr int kQBytes = QREG ? 0 : KS * TERMS * 32 * 16;
  static constexpr int kLdO = DP + 4;                 // of the warps' results, floats
  static constexpr int kRed = kWarps * kRows * (kLdO + 1) * 4;
  static_assert(kRed <= kScales, "the results overlay the rings");
  static constexpr int kSmem = kQ + kQBytes + 1024;
  static constexpr int CTAS = F32Q || DP > 128 ? (DP > 128 ? 1 : 2) : 3;
  static constexpr int VW = DP == 64 ? 8 : 16;        // V bytes of a lane
  static constexpr int VH = DP == 256 ? 2 : 1;        // ... times
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts_f(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// Where chunk ch of a token's row lies in a group's 16 rows, as TMA swizzles them: rows
// of 128 bytes (64 with DP = 64), halves of longer ones one behind the other.  A phase
// of K's reads takes the even or odd chunks of 2 tokens, one of V's 2 chunks of every
// other token of 8: all in different banks.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int token, int ch) {
  if (DP == 64) return token * 64 + ((ch ^ ((token >> 1) & 3)) << 4);
  return (ch >> 3) * (kGroup * 128) + token * 128 + (((ch ^ token) & 7) << 4);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, uint32_t bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// 16 consecutive elements of a query row, from d on, as FP32.
template <bool F32Q>
__device__ __forceinline__ void load_q(const AttnArgs &a, int64_t at, bool on, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  if (!on) return;
  if (F32Q) {
    const float *p = static_cast<const float *>(a.q) + at;
    if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = reinterpret_cast<const float4 *>(p)[i];
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = p[i];
    }
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(a.q) + at;
    if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
          x[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
    }
  }
}

// Puts V's codes that are not finite, of the steps of 32 tokens that a warp went through
// without them, into the results of the rows that see them.
template <int FMT, int DP>
__device__ __noinline__ void put_not_finite(const AttnArgs &a, const Item &it, int first, int all,
                                            int end, float *rows) {
  const Cache &c = a.cache;
#pragma unroll 1
  for (int base = first; base < end; base += kTile) {
    if (base + kStep <= all) continue;
#pragma unroll 1
    for (int t = base; t < min(base + kStep, end); ++t) {
      const int p = divide(t, c.page), page = a.rows.table[it.s * a.rows.ld_table + p];
      if (page < 0 || page >= c.num_pages) continue;
      const uint8_t *v = c.v + it.h * c.head_stride + page * c.page_stride +
                         (t - p * c.page_size) * c.token_stride;
#pragma unroll 1
      for (int d = threadIdx.x & 31; d < c.D; d += 32) {
        if (Format<FMT>::finite(v[d])) continue;
#pragma unroll 1
        for (int r = 0; r < it.rows; ++r)
          if (t < tokens_seen(a, it.q, it.rt * kRows + r)) rows[r * (DP + 4) + d] = NAN;
      }
    }
  }
}

// Four elements of row r, of all warps' results, where some are far below others.
template <int DP>
__device__ __noinline__ float4 join_far(const float *red, const float *red_lse, int r, int d,
                                        float best, float inv) {
  float x[4] = {};
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    const float lse = red_lse[w * kRows + r];
    const bool far = far_below(lse - best);
    const float f = lse == -INFINITY ? 0.0f : ex2(far ? 0.5f * (lse - best) : lse - best);
    const float *p = red + (w * kRows + r) * (DP + 4) + d;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = fmaf(f * inv, far ? p[j] * f : p[j], x[j]);
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}

// Joins what the pieces of a part before this one made with the first warp's results.
template <int DP>
__device__ __noinline__ void join_pieces(const AttnArgs &a, int part, int rows, float *red,
                                         float *red_lse) {
  const int64_t row0 = static_cast<int64_t>(part) * kRows;
  for (int i = threadIdx.x; i < rows * a.cache.D; i += kThreads) {
    const int r = i / a.cache.D, d = i - r * a.cache.D;
    float *p = red + r * (DP + 4) + d;
    *p = joined(weigh(red_lse[r], a.part_lse[row0 + r]), *p, a.part_o[(row0 + r) * DP + d]);
  }
  __syncthreads();
  if (threadIdx.x < rows)
    red_lse[threadIdx.x] = weigh(red_lse[threadIdx.x], a.part_lse[row0 + threadIdx.x]).lse;
  __syncthreads();
}

template <bool F32Q, int FMT, int DP>
__global__ void __launch_bounds__(kThreads, (Cfg<F32Q, DP>::CTAS))
    kv_attention_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ AttnArgs a, const uint64_t timeout_ns) {
  using C = Cfg<F32Q, DP>;
  using Fm = Format<FMT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Share sh;
  __shared__ int64_t warp_sums[kWarps];
  __shared__ Walk walk;
  __shared__ Item it;
  __shared__ int more;
  __shared__ volatile int abort_flag;
  const uint32_t raw = smem_addr(smem_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t *const smem = smem_raw + (sbase - raw);
  // The same in all lanes, which the compiler would not see otherwise.
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t bars = sbase + C::kBar + warp * kStages * 8;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
    abort_flag = 0;
  }
  if (!a.late) pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) a.desc[blockIdx.x].parts = 0;
  share_out<kThreads, kRows, kTile, kItemCost>(a, &sh, warp_sums);
  const Cache &kc = a.cache;
  const uint32_t ring = sbase + warp * C::kRing;
  const uint32_t scale_ring = sbase + C::kScales + warp * kStages * C::kScaleStage;
  const uint32_t qsm = sbase + C::kQ;
  uint32_t put = 0, taken = 0;         // groups requested and taken so far
  auto el = [](int f, int c) {         // first element of a lane's chunk f of K's rows
    return DP == 64 ? 16 * c : (f >> 1) * 128 + 32 * c + 16 * (f & 1);
  };

  if (threadIdx.x == 0) start_walk<kRows>(a, sh, &walk);
  for (;;) {
    if (threadIdx.x == 0) more = next_item<kRows, kTile, kItemCost, kWarps * kPiece>(a, &walk, &it);
    __syncthreads();
    if (!more) break;
    const Seq q = it.q;
    const int s = it.s, h = it.h, rt = it.rt, tile0 = it.tile0, count = it.count, rows = it.rows;

    // This lane's rows are rt * 16 + g and that + 8; they see the tokens below
    // seen[0] and seen[1].  Tokens from `all` on are not seen by every row.
    int tok[2], head[2], seen[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rt * kRows + min(g + 8 * i, rows - 1);
      tok[i] = divide(r, a.group);
      head[i] = h * a.G + r - tok[i] * a.G;
      seen[i] = g + 8 * i < rows ? tokens_seen(a, q, r) : 0;
    }
    const int all = tokens_seen(a, q, rt * kRows);
    const int most = tokens_seen(a, q, rt * kRows + rows - 1);
    const int begin = tile0 * kTile, end = min(begin + count * kTile, most);

    // Pages are looked up one step before they are needed.  Where pages are made of
    // whole groups, a group is two copies by TMA (a page that there is not: zeros);
    // else each row is copied in chunks of 16 bytes.
    const int32_t *table = a.rows.table + s * a.rows.ld_table;
    const uint8_t *kbase = kc.k + h * kc.head_stride, *vbase = kc.v + h * kc.head_stride;
    const float *ksbase = kc.k_scale + h * kc.scale_head_stride;
    const float *vsbase = kc.v_scale + h * kc.scale_head_stride;
    auto page_at = [&](int first) {
      const int t = first + lane;
      return t < end ? table[divide(t, kc.page)] : -1;
    };
    auto request = [&](int first, int page) {
      const int t = first + lane;
      bool on = t < end;
      if (on && (page < 0 || page >= kc.num_pages)) {
        atomicOr(a.rows.status, kStatusBadDeviceArg);
        on = false;
      }
      const int place = t - divide(t, kc.page) * kc.page_size;
      const int slot = put % kStages;
      const uint32_t dst = ring + slot * C::kStage, bar = bars + 8 * slot;
      const uint32_t sdst = scale_ring + slot * C::kScaleStage + lane * 4;
      const int64_t sc = on ? page * kc.scale_page_stride + place * kc.scale_token_stride : 0;
      cp_async4(sdst, ksbase + sc, on);
      cp_async4(sdst + 4 * kStep, vsbase + sc, on);
      if (a.tma) {
        // Every lane has read the slot before the barrier that ended its turn.
        if (lane == 0) mbar_arrive_expect_tx(bar, C::kStage);
        __syncwarp();
        if (lane % kGroup == 0) {
          const int p = on ? page : kc.num_pages;
          const uint32_t at = dst + lane / kGroup * 2 * C::kK;
#pragma unroll
          for (int f = 0; f < C::VH; ++f) {
            tma_load_4d(at + f * kGroup * 128, &tmK, bar, 128 * f, place, h, p);
            tma_load_4d(at + C::kK + f * kGroup * 128, &tmV, bar, 128 * f, place, h, p);
          }
        }
      } else {
        const int64_t code = on ? page * kc.page_stride + place * kc.token_stride : -1;
#pragma unroll 1
        for (int i = 0; i < kStep * C::CH / 32; ++i) {
          const int id = lane + 32 * i, token = id / C::CH, ch = id % C::CH;
          const int64_t off = __shfl_sync(0xffffffffu, code, token);
          const bool ok = off >= 0 && ch * 16 < kc.D;
          const int64_t from = ok ? off + ch * 16 : 0;
          const uint32_t at = dst + token / kGroup * 2 * C::kK + chunk_at<DP>(token % kGroup, ch);
          cp_async16(at, kbase + from, ok);
          cp_async16(at + C::kK, vbase + from, ok);
        }
      }
      ++put;
    };
    const int first = begin + warp * kStep;
    int page = page_at(first);
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
      if (first + i * kTile < end) {
        const int p = page;
        page = page_at(first + (i + 1) * kTile);
        request(first + i * kTile, p);
      }
      cp_commit();
    }

    // Query fragments: k 2c, 2c+1, 2c+8, 2c+9 of step 4 f + j stand for the elements
    // el(f, c) + 4 j .. + 3, so that a lane's codes are 16 bytes of a row.
    uint32_t qf[C::QREG ? C::KS * C::TERMS : 1][4];
    float factor[2];
    {
      int e[2];
      int64_t at[2];
      float m[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 2; ++i)
        at[i] = (static_cast<int64_t>(q.row0) + tok[i]) * a.ldq + head[i] * a.ldq_head;
      float all_x[DP / 64][2][16];
#pragma unroll
      for (int f = 0; f < DP / 64; ++f)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          load_q<F32Q>(a, at[i] + el(f, c), el(f, c) < kc.D, all_x[f][i]);
#pragma unroll
          for (int j = 0; j < 16; ++j) m[i] = fmaxf(m[i], fabsf(all_x[f][i][j]));
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
        m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
        e[i] = min(max(8 - exponent_of(m[i]), -126), 126);
        factor[i] = power_of_two(-e[i]) * a.scale_log2;
      }
#pragma unroll
      for (int f = 0; f < DP / 64; ++f) {
        float(&x)[2][16] = all_x[f];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float up = power_of_two(e[i]);
#pragma unroll
          for (int j = 0; j < 16; ++j) x[i][j] *= up;
        }
#pragma unroll
        for (int t = 0; t < C::TERMS; ++t) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float *p = &x[k & 1][4 * j + (k >> 1) * 2];
              w[k] = pack_half(p[0], p[1]);
              if (t + 1 < C::TERMS) {
                const float2 r = half2_floats(w[k]);
                p[0] -= r.x;
                p[1] -= r.y;
              }
            }
            const int step = (4 * f + j) * C::TERMS + t;
            if (C::QREG) {
#pragma unroll
              for (int k = 0; k < 4; ++k) qf[step][k] = w[k];
            } else if (warp == 0) {
              st_shared_v4(qsm + (step * 32 + lane) * 16, w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      if (!C::QREG) __syncthreads();
    }

    float o[C::VH * C::VW][4];
#pragma unroll
    for (int j = 0; j < C::VH * C::VW; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
    float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float far_top[2] = {-INFINITY, -INFINITY}, far_sum[2] = {0.0f, 0.0f};  // see kSpan
    int e0 = 0;
    bool poison = false;
    // Tokens whose shares are added up beside are rare: the loop stands here twice, first
    // without the code for them, which would be fetched past in every turn (256 requests of
    // 1024 tokens 128 us with it), and then with it, from a step with such tokens on, of which
    // `done` parts are done, to one without; the second time to the end.  The same requests
    // take 114 us, with one such token in each 136 (171 if the first time were to the end),
    // with a tenth of all tokens 222 (169).
    int base = first, done = 0;
    bool alive = true, back = true;
    do {
#pragma unroll
      for (int rare = 0; rare < 2; ++rare) {
#pragma unroll 1
        for (; alive && base < end; base += kTile) {
          if (!rare || done == 0) {
            cp_wait<kStages - 2>();
            if (a.tma)
              alive = __all_sync(0xffffffffu,
                                 mbar_wait(bars + 8 * (taken % kStages), (taken / kStages) & 1u,
                                           timeout_ns, a.rows.status, &abort_flag));
            if (!alive) break;
            ++taken;
            __syncwarp();
            const int ahead = base + (kStages - 1) * kTile;
            if (ahead < end) {
              const int p = page;
              page = page_at(ahead + kTile);
              request(ahead, p);
            }
            cp_commit();
          }
          const int slot = (taken - 1) % kStages;
          const uint32_t st = ring + slot * C::kStage, scales = scale_ring + slot * C::kScaleStage;
          // V's scales: logarithm and reciprocal, relative to a power of two near the first.
          if (base == first && (!rare || done == 0)) {
            e0 = min(exponent_of(lds_f(scales + 4 * kStep)), 126);
            __syncwarp();
          }
          uint32_t far = 0;  // tokens whose shares are added up beside
          bool some = false;
          if (!rare || done < 2) {
            const float v = lds_f(scales + 4 * (kStep + lane));
            const bool fine = base + lane < end && v > 0.0f && v < INFINITY;
            // Whether the exponent (of subnormal numbers one less than exponent_of) is within
            // e0 - kSpan .. e0 + kSpan.
            const uint32_t above = (__float_as_uint(v) >> 23) - static_cast<uint32_t>(e0 + 127 - kSpan);
            if (__any_sync(0xffffffffu, fine && above > 2 * kSpan)) {
              if (!rare) {
                done = 1;
                break;
              }
              const int top = __reduce_max_sync(0xffffffffu, fine ? min(exponent_of(v), 126) : -126);
              if (top > e0 + kSpan) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  add_share(far_top[k], far_sum[k], M[k] - kShift, l[k]);
                  l[k] = 0.0f;
                  M[k] -= static_cast<float>(top - e0);
                }
                e0 = top;
              }
              far = __ballot_sync(0xffffffffu, fine && exponent_of(v) < e0 - kSpan);
            }
            const float near = v * power_of_two(-e0);
            const bool less = far >> lane & 1;
            sts_f(scales + 4 * (kStep + lane), base + lane >= end ? 0.0f
                                               : !fine            ? NAN
                                               : less             ? log2_far(v, e0)
                                                                  : lg2(near));
            // A bad scale is in the exponent alone: rows that do not see it have weight 0.
            sts_f(scales + 4 * (2 * kStep + lane), !fine ? 1.0f : less ? 0.0f : rcp(near));
          }
          // What lies behind the end may be anything.  Where some rows do not see a token (weight
          // 0), its codes of V that are not finite must not reach them: they are taken out and put
          // in at the end.
          const bool partial = all < most && base + kStep > all;
          if (partial || base + kStep > end) {
            const uint32_t row = st + (lane / kGroup * 2 + 1) * C::kK;
#pragma unroll 1
            for (int ch = 0; ch < C::CH; ++ch) {
              const uint32_t at = row + chunk_at<DP>(lane % kGroup, ch);
              const uint4 v = lds128(at);
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (base + lane >= end) w[j] = 0;
                if (partial) poison |= Fm::clear4(w[j]);
              }
              st_shared_v4(at, w[0], w[1], w[2], w[3]);
            }
          }
          // Scores of tokens 16 u + 8 i + g against the 16 rows, in sc[2 u + i].
          float sc[2 * kSubs][4] = {};
#pragma unroll
          for (int u = 0; u < kSubs; ++u) {
#pragma unroll
            for (int f = 0; f < DP / 64; ++f) {
              uint32_t kw[2][4];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint4 w = lds128(st + u * 2 * C::kK + chunk_at<DP>(g + 8 * i, el(f, c) / 16));
                kw[i][0] = w.x; kw[i][1] = w.y; kw[i][2] = w.z; kw[i][3] = w.w;
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t b[2][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  b[i][0] = decode2<FMT>(kw[i][j] & 0xffffu);
                  b[i][1] = decode2<FMT>(kw[i][j] >> 16);
                }
#pragma unroll
                for (int t = 0; t < C::TERMS; ++t) {
                  const int step = (4 * f + j) * C::TERMS + t;
                  if (C::QREG) {
                    mma_f16(sc[2 * u], qf[step], b[0][0], b[0][1]);
                    mma_f16(sc[2 * u + 1], qf[step], b[1][0], b[1][1]);
                  } else {
                    const uint4 w = lds128(qsm + (step * 32 + lane) * 16);
                    const uint32_t qw[4] = {w.x, w.y, w.z, w.w};
                    mma_f16(sc[2 * u], qw, b[0][0], b[0][1]);
                    mma_f16(sc[2 * u + 1], qw, b[1][0], b[1][1]);
                  }
                }
              }
            }
          }
          __syncwarp();
          // Adds up beside the shares of the tokens in `mask`, whose scores x(i, k) gives.
          auto set_aside = [&](uint32_t mask, auto score) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float x[4 * kSubs], top = -INFINITY;
#pragma unroll
              for (int i = 0; i < 4 * kSubs; ++i) {
                const int t = 8 * (i >> 1) + 2 * c + (i & 1);
                x[i] = (mask >> t & 1) && base + t < seen[k] ? score(sc[i >> 1][2 * k + (i & 1)], t, k)
                                                             : -INFINITY;
                top = fmaxf(top, x[i]);
              }
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
              // The row's four lanes have the same maximum and a part of the sum each.
              const float from = top == -INFINITY ? 0.0f : top;
              float sum = 0.0f;
#pragma unroll
              for (int i = 0; i < 4 * kSubs; ++i) sum += ex2(x[i] - from);
              add_share(far_top[k], far_sum[k], top, sum);
            }
          };
          if (rare && far)
            set_aside(far, [&](float s, int t, int k) { return s * lds_f(scales + 4 * t) * factor[k]; });
          // Exponents and weights of tokens 8 i + 2c, 8 i + 2c + 1.
#pragma unroll
          for (int i = 0; i < 2 * kSubs; ++i) {
            const float2 ks = lds_f2(scales + 32 * i + 8 * c);
            const float2 lv = lds_f2(scales + 4 * kStep + 32 * i + 8 * c);
            sc[i][0] = fmaf(sc[i][0] * ks.x, factor[0], lv.x);
            sc[i][1] = fmaf(sc[i][1] * ks.y, factor[0], lv.y);
            sc[i][2] = fmaf(sc[i][2] * ks.x, factor[1], lv.x);
            sc[i][3] = fmaf(sc[i][3] * ks.y, factor[1], lv.y);
          }
          if (base + kStep > min(all, end)) {
#pragma unroll
            for (int i = 0; i < 2 * kSubs; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (base + 8 * i + 2 * c + (k & 1) >= min(seen[k >> 1], end)) sc[i][k] = -INFINITY;
          }
          float mx[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            mx[k] = fmaxf(sc[0][2 * k], sc[0][2 * k + 1]);
#pragma unroll
            for (int i = 1; i < 2 * kSubs; ++i) mx[k] = fmaxf(mx[k], fmaxf(sc[i][2 * k], sc[i][2 * k + 1]));
          }
          if (__any_sync(0xffffffffu, mx[0] > M[0] + kLazy || mx[1] > M[1] + kLazy)) {
            // A row of zeros in V adds nothing to the result, whatever its scale: it must not
            // take the others' weights towards a half's end.  Nearly all have another code
            // among the first 16.
            uint32_t zeros = base + kStep <= end ? 0xffffffffu : (1u << (end - base)) - 1;
#pragma unroll 1
            for (int ch = 0; ch < C::CH && zeros != 0; ++ch) {
              const uint4 w = lds128(st + (lane / kGroup * 2 + 1) * C::kK +
                                     chunk_at<DP>(lane % kGroup, ch));
              zeros &= __ballot_sync(0xffffffffu, ((w.x | w.y | w.z | w.w) & 0x7f7f7f7fu) == 0);
            }
            if (zeros && !rare) {
              done = 2;
              break;
            }
            some = zeros != 0;
            if (rare && zeros) {
              set_aside(zeros & ~far,
                        [&](float s, int t, int) { return s - lds_f(scales + 4 * (kStep + t)); });
              mx[0] = mx[1] = -INFINITY;
#pragma unroll
              for (int i = 0; i < 2 * kSubs; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (zeros >> (8 * i + 2 * c + (k & 1)) & 1) sc[i][k] = -INFINITY;
                  mx[k >> 1] = fmaxf(mx[k >> 1], sc[i][k]);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float m = mx[k];
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
              m = fmaxf(m, M[k]);
              const float down = m == -INFINITY ? 1.0f : ex2(M[k] - m);
              M[k] = m;
              l[k] *= down;
#pragma unroll
              for (int j = 0; j < C::VH * C::VW; ++j) {
                o[j][2 * k] *= down;
                o[j][2 * k + 1] *= down;
              }
            }
          }
          const float top[2] = {M[0] == -INFINITY ? 0.0f : M[0] - kShift,
                                M[1] == -INFINITY ? 0.0f : M[1] - kShift};
          uint32_t pf[kSubs][4];
#pragma unroll
          for (int i = 0; i < 2 * kSubs; ++i) {
            const float2 iv = lds_f2(scales + 8 * kStep + 32 * i + 8 * c);
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[i][k] = ex2(sc[i][k] - top[k >> 1]);
            l[0] = fmaf(sc[i][0], iv.x, fmaf(sc[i][1], iv.y, l[0]));
            l[1] = fmaf(sc[i][2], iv.x, fmaf(sc[i][3], iv.y, l[1]));
            pf[i >> 1][2 * (i & 1)] = pack_half(sc[i][0], sc[i][1]);
            pf[i >> 1][2 * (i & 1) + 1] = pack_half(sc[i][2], sc[i][3]);
          }
          // Values.
#pragma unroll
          for (int u = 0; u < kSubs; ++u) {
#pragma unroll
            for (int f = 0; f < C::VH; ++f) {
              uint32_t vw[4][C::VW / 4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int token = 2 * c + (i & 1) + 8 * (i >> 1);
                const uint32_t v_at = st + u * 2 * C::kK + C::kK;
                if (C::VW == 16) {
                  const uint4 v = lds128(v_at + chunk_at<DP>(token, 8 * f + g));
                  vw[i][0] = v.x; vw[i][1] = v.y; vw[i][C::VW / 8] = v.z; vw[i][C::VW / 4 - 1] = v.w;
                } else {
                  const uint2 v = lds64(v_at + chunk_at<DP>(token, g >> 1) + (g & 1) * 8);
                  vw[i][0] = v.x; vw[i][1] = v.y;
                }
              }
#pragma unroll
              for (int j = 0; j < C::VW / 4; ++j) {
                const uint32_t a0 = __byte_perm(vw[0][j], vw[1][j], 0x5140);
                const uint32_t a1 = __byte_perm(vw[0][j], vw[1][j], 0x7362);
                const uint32_t b0 = __byte_perm(vw[2][j], vw[3][j], 0x5140);
                const uint32_t b1 = __byte_perm(vw[2][j], vw[3][j], 0x7362);
                float(*oo)[4] = &o[f * C::VW + 4 * j];
                mma_f16(oo[0], pf[u], decode2<FMT>(a0 & 0xffffu), decode2<FMT>(b0 & 0xffffu));
                mma_f16(oo[1], pf[u], decode2<FMT>(a0 >> 16), decode2<FMT>(b0 >> 16));
                mma_f16(oo[2], pf[u], decode2<FMT>(a1 & 0xffffu), decode2<FMT>(b1 & 0xffffu));
                mma_f16(oo[3], pf[u], decode2<FMT>(a1 >> 16), decode2<FMT>(b1 >> 16));
              }
            }
          }
          // Reads before the copies that a next turn asks for.
          if (a.tma) fence_proxy_async_smem();
          if (rare) {
            done = 0;
            if (back && !some && far == 0) {
              back = false;
              base += kTile;
              break;
            }
          }
        }
      }
    } while (alive && base < end);
    cp_wait<0>();
    for (; taken < put; ++taken)  // where a wait ran out
      if (a.tma)
        mbar_wait_drain(bars + 8 * (taken % kStages), (taken / kStages) & 1u, timeout_ns,
                        a.rows.status);

    // Each warp's result, normalised, with its logarithm (base 2); then all four's.
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);
    float *red_lse = red + kWarps * kRows * C::kLdO;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float sum = l[k], beside = far_sum[k];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      beside += __shfl_xor_sync(0xffffffffu, beside, 1);
      beside += __shfl_xor_sync(0xffffffffu, beside, 2);
      const Total all_of = total_of(M[k] - kShift, sum, far_top[k], beside, e0);
      float *row = red + (warp * kRows + g + 8 * k) * C::kLdO;
#pragma unroll
      for (int j = 0; j < C::VH * C::VW; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          row[j / C::VW * 128 + (2 * c + i) * C::VW + j % C::VW] =
              o[j][2 * k + i] * all_of.f0 * all_of.f1;
      if (c == 0) red_lse[warp * kRows + g + 8 * k] = all_of.lse;
    }
    if (__any_sync(0xffffffffu, poison)) {
      __syncwarp();
      put_not_finite<FMT, DP>(a, it, first, all, end, red + warp * kRows * C::kLdO);
    }
    __syncthreads();
    if (a.late) pdl_wait();  // the prefix's results
    const bool whole = it.first == 0 && tile0 + count == it.tiles;
    const int part = 2 * blockIdx.x + (it.first > 0 ? 0 : 1);
    if (it.after) join_pieces<DP>(a, part, rows, red, red_lse);
    constexpr int kPieces = DP / 8;
    for (int i = threadIdx.x; i < rows * kPieces; i += kThreads) {
      const int r = i / kPieces, d = i % kPieces * 8;
      float lse[kWarps], best = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        lse[w] = red_lse[w * kRows + r];
        best = fmaxf(best, lse[w]);
      }
      // A NaN is in no maximum, but in its weight.
      float weight[kWarps], sum = 0.0f;
      bool far = false;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        weight[w] = lse[w] == -INFINITY ? 0.0f : ex2(lse[w] - best);
        sum += weight[w];
        far |= far_below(lse[w] - best);
      }
      const float inv = sum == 0.0f ? 0.0f : rcp(sum);
      const float all_lse = sum == 0.0f ? -INFINITY : best + lg2(sum);
      float x[8] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {  // 0 x NaN too: a V that is not finite
        const float *p = red + (w * kRows + r) * C::kLdO + d;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(weight[w] * inv, p[j], x[j]);
      }
      if (far) {
        const float4 lo = join_far<DP>(red, red_lse, r, d, best, inv);
        const float4 hi = join_far<DP>(red, red_lse, r, d + 4, best, inv);
        x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
        x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
      }
      if (d >= kc.D) continue;
      if (whole) {
        const int rr = rt * kRows + r, t = divide(rr, a.group);
        const int64_t row = static_cast<int64_t>(q.row0) + t;
        const int hq = h * a.G + rr - t * a.G;
        emit<8>(a, row, hq, d, x, all_lse, weigh(a, row, hq, all_lse));
      } else {
        float *p = a.part_o + (static_cast<int64_t>(part) * kRows + r) * DP + d;
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
        if (d == 0) a.part_lse[part * kRows + r] = all_lse;
      }
    }
    if (threadIdx.x == 0 && !whole && !it.more && it.first == 0)
      a.desc[blockIdx.x] = {s, h, rt, owner_of(sh, it.end - 1) - static_cast<int>(blockIdx.x) + 1};
    fence_proxy_async_smem();
    __syncthreads();  // the results overlay the rings
    if (abort_flag) break;
  }
  if (a.late) pdl_wait();  // who waits for this kernel waits for the one before it
}

// ---------------------------------------------------------------------- join
// Joins the partial results of items that several CTAs shared: CTA b began it
// (its second partial result), the next parts - 1 went on (their first ones).  Where
// parts are few, which is what a boundary between two CTAs makes, a warp takes a few
// rows at once; else a row has one warp or several, whose sums are added in order.
// Both kernels' items are joined in one launch.
//
// Bound: latency, as most of it is a chain of loads (what there is to join, whose rows,
// their logarithms, the parts).  A row at a time of each warp took 22 us behind two
// prompts of 2048 tokens (150 items of two parts, 256 rows each), 18 behind 6 ragged
// ones and 13 behind one sequence of 131072 tokens (8 items of 57 parts); this 12, 8 and
// 7.  The grid: with 3, 4, 6 or 8 CTAs an SM 64 requests take 108, 120, 117, 106 us a
// call in a graph and 120, 146, 143, 108 called one by one (why so much more was not
// found; without the join it is 102), one request of 2048 tokens 15.8, 15.8, 15.8, 17.1.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kFewParts = 4;
constexpr int kManyParts = 16;
constexpr int kJoinResident = 3;  // CTAs of an SM at once, 2 with heads above 128
constexpr int kJoinCtasPerSm = 8;
constexpr int kAtOnce = 4;      // parts whose loads are under way

struct JoinSide {
  const float *part_o, *part_lse;
  const Desc *desc;
  int32_t BM, ctas, blocks;  // blocks for each CTA
};

// V floats, 4 V-byte aligned.
template <int V>
__device__ __forceinline__ void load_part(const float *p, float (&y)[V]) {
  if (V >= 4) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(p + j);
      y[j] = f.x; y[j + 1] = f.y; y[V >= 4 ? j + 2 : 0] = f.z; y[V >= 4 ? j + 3 : 0] = f.w;
    }
  } else {
    const float2 f = *reinterpret_cast<const float2 *>(p);
    y[0] = f.x; y[1] = f.y;
  }
}

template <int DP>
__global__ void __launch_bounds__(kJoinThreads, DP > 128 ? 2 : kJoinResident)
    kv_join_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ JoinSide few,
                   const __grid_constant__ JoinSide many) {
  constexpr int V = DP / 32;
  constexpr int R = DP > 128 ? 2 : 4;   // rows of a warp at once, where parts are few
  __shared__ float sums[kJoinWarps][DP + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int few_blocks = few.ctas * few.blocks;
  const int blocks = few_blocks + many.ctas * many.blocks;
  // A few rows of a CTA's item in each turn.  Most have nothing to join, and CTAs that
  // have are about equally far apart: a grid of an odd size deals them out.
  auto turn_of = [&](int block, bool *first, int *cta) {
    *first = block < few_blocks;
    const int at = *first ? block : block - few_blocks, ctas = *first ? few.ctas : many.ctas;
    *cta = at % ctas;
    return at / ctas;
  };
  // Each lane looks at one of the next 32 turns.
  for (int round = 0; blockIdx.x + round * gridDim.x < blocks; round += 32) {
    const int64_t mine = blockIdx.x + static_cast<int64_t>(round + lane) * gridDim.x;
    Desc look = {0, 0, 0, 0};
    if (mine < blocks) {
      bool first;
      int cta;
      const int turn = turn_of(static_cast<int>(mine), &first, &cta);
      look = (first ? few.desc : many.desc)[cta];
      const int group = look.parts <= kFewParts ? kJoinWarps * R : first ? 1 : kJoinWarps;
      if (turn * group >= (first ? few.BM : many.BM)) look.parts = 0;
    }
    for (uint32_t some = __ballot_sync(0xffffffffu, look.parts > 0); some; some &= some - 1) {
      const int i = __ffs(some) - 1;
      const Desc d = {__shfl_sync(0xffffffffu, look.s, i), __shfl_sync(0xffffffffu, look.h, i),
                      __shfl_sync(0xffffffffu, look.rt, i), __shfl_sync(0xffffffffu, look.parts, i)};
      bool first;
      int cta;
      const int turn = turn_of(blockIdx.x + (round + i) * gridDim.x, &first, &cta);
      const float *part_o = first ? few.part_o : many.part_o;
      const float *part_lse = first ? few.part_lse : many.part_lse;
      const int BM = first ? few.BM : many.BM;
      const Seq q = load_seq(a, d.s);
      const int rows = min(BM, q.n * a.G - d.rt * BM);
      if (d.parts <= kFewParts) {
        const int r0 = (turn * kJoinWarps + warp) * R;
        if (r0 >= rows) continue;
        auto part = [&](int i) {
          return static_cast<int64_t>(2 * (cta + i) + (i == 0 ? 1 : 0)) * BM + r0;
        };
        // Lane 4 u + i: part i of row u.
        const int own = lane & 3, row = (lane >> 2) % R;
        const float lse =
            own < d.parts && r0 + row < rows ? part_lse[part(own) + row] : -INFINITY;
        float x[R][V] = {}, all_lse = -INFINITY;
        float weight = 0.0f, half = 1.0f;  // `half` where a part is far below
        bool far = false;
#pragma unroll 1
        for (int i0 = 0; i0 < d.parts; i0 += 2) {
          float y[R][2][V];
#pragma unroll
          for (int u = 0; u < R; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const bool on = r0 + u < rows && i0 + k < d.parts;
              const float *p = part_o + (part(i0 + k) + u) * DP + lane * V;
#pragma unroll
              for (int j = 0; j < V; ++j) y[u][k][j] = 0.0f;
              if (on) load_part<V>(p, y[u][k]);
            }
          if (i0 == 0) {  // weights, while the first parts come
            float best = lse;
            best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
            best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
            const float w = lse == -INFINITY ? 0.0f : ex2(lse - best);
            far = __any_sync(0xffffffffu, far_below(lse - best));
            float sum = w;
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            weight = sum == 0.0f ? 0.0f : w * rcp(sum);
            if (far_below(lse - best)) {
              half = ex2(0.5f * (lse - best));
              weight = half * rcp(sum);
            }
            all_lse = sum == 0.0f ? -INFINITY : best + lg2(sum);
          }
#pragma unroll
          for (int u = 0; u < R; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float w = __shfl_sync(0xffffffffu, weight, 4 * u + i0 + k);
              if (far) {
                const float f = __shfl_sync(0xffffffffu, half, 4 * u + i0 + k);
#pragma unroll
                for (int j = 0; j < V; ++j) y[u][k][j] *= f;
              }
#pragma unroll
              for (int j = 0; j < V; ++j) x[u][j] = fmaf(w, y[u][k][j], x[u][j]);
            }
        }
#pragma unroll
        for (int u = 0; u < R; ++u) {
          const float l = __shfl_sync(0xffffffffu, all_lse, 4 * u);
          if (r0 + u >= rows || lane * V >= a.cache.D) continue;
          const int rr = d.rt * BM + r0 + u, t = divide(rr, a.group);
          const int64_t row = static_cast<int64_t>(q.row0) + t;
          const int hq = d.h * a.G + rr - t * a.G;
          emit<V>(a, row, hq, lane * V, x[u], l, weigh(a, row, hq, l));
        }
        continue;
      }
      const int group = first ? 1 : kJoinWarps;                 // rows of this turn
      const int each = d.parts > kManyParts ? min(group, 2) : group;  // rows at a time
      const int warps = kJoinWarps / each;                      // of a row
      const int r_end = min(rows, (turn + 1) * group);
      for (int r0 = turn * group; r0 < r_end; r0 += each) {
        const int r = r0 + warp / warps, rr = d.rt * BM + r;
        const bool on = r < r_end;
        auto part = [&](int i) {
          return static_cast<int64_t>(2 * (cta + i) + (i == 0 ? 1 : 0)) * BM + r;
        };
        float best = -INFINITY, x[V] = {}, sum = 0.0f;
        if (on) {
          for (int i = lane; i < d.parts; i += 32) best = fmaxf(best, part_lse[part(i)]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
          const int i1 = d.parts * (warp % warps + 1) / warps;
          for (int i0 = d.parts * (warp % warps) / warps; i0 < i1; i0 += 32) {
            // A weight to each lane, so that the parts' loads wait for nothing.
            const int n = min(32, i1 - i0);
            const float lse = lane < n ? part_lse[part(i0 + lane)] : -INFINITY;
            float mine = lse == -INFINITY ? 0.0f : ex2(lse - best), half = 1.0f;
            if (far_below(lse - best)) mine = half = ex2(0.5f * (lse - best));
            const bool far = __any_sync(0xffffffffu, half < 1.0f);
#pragma unroll 1
            for (int i = 0; i < n; i += kAtOnce) {
              float y[kAtOnce][V];
#pragma unroll
              for (int u = 0; u < kAtOnce; ++u)
                load_part<V>(part_o + part(i0 + min(i + u, n - 1)) * DP + lane * V, y[u]);
#pragma unroll
              for (int u = 0; u < kAtOnce; ++u) {
                if (i + u >= n) break;
                const float w = __shfl_sync(0xffffffffu, mine, i + u);
                float f = 1.0f;
                if (far) {
                  f = __shfl_sync(0xffffffffu, half, i + u);
#pragma unroll
                  for (int j = 0; j < V; ++j) y[u][j] *= f;
                }
                sum = fmaf(w, f, sum);
#pragma unroll
                for (int j = 0; j < V; ++j) x[j] = fmaf(w, y[u][j], x[j]);
              }
            }
          }
        }
        if (warps > 1) {
          __syncthreads();
#pragma unroll
          for (int j = 0; j < V; ++j) sums[warp][lane * V + j] = x[j];
          if (lane == 0) sums[warp][DP] = sum;
          __syncthreads();
          if (warp % warps > 0) continue;
          for (int w = warp + 1; w < warp + warps; ++w) {
            sum += sums[w][DP];
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] += sums[w][lane * V + j];
          }
        }
        if (on && lane * V < a.cache.D) {
          const float inv = sum == 0.0f ? 0.0f : rcp(sum);
#pragma unroll
          for (int j = 0; j < V; ++j) x[j] *= inv;
          const float lse = sum == 0.0f ? -INFINITY : best + lg2(sum);
          const int t = divide(rr, a.group);
          const int64_t row = static_cast<int64_t>(q.row0) + t;
          const int hq = d.h * a.G + rr - t * a.G;
          emit<V>(a, row, hq, lane * V, x, lse, weigh(a, row, hq, lse));
        }
      }
    }
  }
}

template <typename Kern, typename... Args>
fp8la_status launch(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t s,
                    const Args &...a) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a...) == cudaSuccess ? FP8LA_OK : FP8LA_ERR_CUDA;
}

// Codes as [page][head][place][D] in boxes of 16 places and up to 128 bytes.  A
// dimension of one element has a stride of no meaning, for which TMA gets another one.
bool code_map(CUtensorMap *m, const uint8_t *p, const Cache &c, int DP) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.heads),
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {
      static_cast<cuuint64_t>(c.page_size > 1 ? c.token_stride : 256),
      static_cast<cuuint64_t>(c.heads > 1 ? c.head_stride : 256),
      static_cast<cuuint64_t>(c.num_pages > 1 ? c.page_stride : 256)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(DP < 128 ? DP : 128), kGroup, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(p), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             DP == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F32Q, int FMT, int DP>
fp8la_status launch_few_one(AttnArgs a, int slot, int ctas, cudaStream_t s) {
  using C = Cfg<F32Q, DP>;
  auto kern = kv_attention_kernel<F32Q, FMT, DP>;
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::kSmem);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  // TMA's limits: strides below 2^40 bytes.  Measured, 64 sequences of 8192 tokens: 179
  // us with TMA, 193 with pages of 24, which are copied in chunks of 16 bytes (181, 198 since).
  CUtensorMap k = {}, v = {};
  const int64_t most = int64_t(1) << 40;
  a.tma = a.cache.page_size % kGroup == 0 && a.cache.page_stride < most &&
          a.cache.head_stride < most && a.cache.token_stride < most &&
          code_map(&k, a.cache.k, a.cache, DP) && code_map(&v, a.cache.v, a.cache, DP);
  return launch(kern, dim3(ctas), kThreads, C::kSmem, s, k, v, a, wait_timeout_ns());
}

int padded_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// CTAs of the few-row kernel on the device.
int few_ctas(bool f32, int DP) {
  const int n = sm_count();
  const int per = DP == 64 ? (f32 ? Cfg<true, 64>::CTAS : Cfg<false, 64>::CTAS)
                  : DP == 128 ? (f32 ? Cfg<true, 128>::CTAS : Cfg<false, 128>::CTAS)
                              : (f32 ? Cfg<true, 256>::CTAS : Cfg<false, 256>::CTAS);
  return (n > 0 ? n : 1) * per;
}

template <bool F32Q, int FMT>
fp8la_status launch_few_fmt(const AttnArgs &a, int DP, int slot, int ctas, cudaStream_t s) {
  if (DP == 64) return launch_few_one<F32Q, FMT, 64>(a, slot, ctas, s);
  if (DP == 128) return launch_few_one<F32Q, FMT, 128>(a, slot + 1, ctas, s);
  return launch_few_one<F32Q, FMT, 256>(a, slot + 2, ctas, s);
}

fp8la_status launch_few(const AttnArgs &a, bool f32, int format, int ctas, cudaStream_t s) {
  const int DP = padded_dim(a.cache.D);
  if (f32)
    return format == FP8LA_FORMAT_E4M3 ? launch_few_fmt<true, 0>(a, DP, 80, ctas, s)
                                       : launch_few_fmt<true, 1>(a, DP, 83, ctas, s);
  return format == FP8LA_FORMAT_E4M3 ? launch_few_fmt<false, 0>(a, DP, 86, ctas, s)
                                     : launch_few_fmt<false, 1>(a, DP, 89, ctas, s);
}

// CTAs of the many-row kernel.
int many_ctas() {
  const int n = sm_count();
  return n > 0 ? n : 1;
}

// Workspace: each kernel's partial results and their descriptions, then the prefix's
// results.
struct Part {
  int64_t o, lse, desc;
};
struct Layout {
  Part few, many;
  int64_t raw_o, raw_lse, bytes;
};
Layout layout_of(int64_t T, int Hq, int D, bool prefix) {
  Layout l;
  int64_t at = 0;
  auto take = [&](int64_t n) {
    const int64_t p = at;
    at += (n + 255) / 256 * 256;
    return p;
  };
  const int DP = padded_dim(D);
  auto part = [&](int64_t ctas, int64_t BM) {
    Part p;
    p.o = take(2 * ctas * BM * DP * 4);
    p.lse = take(2 * ctas * BM * 4);
    p.desc = take(ctas * static_cast<int64_t>(sizeof(Desc)));
    return p;
  };
  l.few = part(few_ctas(false, DP), kRows);
  l.many = part(DP <= 128 ? many_ctas() : 0, kManyItemRows);
  l.raw_o = take(prefix ? T * Hq * D * 4 : 0);
  l.raw_lse = take(prefix ? T * Hq * 4 : 0);
  l.bytes = at + 256 - 16;  // begins at a multiple of 256, wherever the caller's does
  return l;
}

// Rows (tokens times heads of a group) of a sequence up to which it takes mma.sync.
// Measured, us, mma.sync / tcgen05, 8 K/V heads of 128: 16 sequences of 4000 tokens with
// 32 rows 65 / 101, 64 rows 105 / 103, 128 rows 182 / 108; one of 8000 tokens with 64 rows
// 34 / 41, 128 rows 42 / 42; 64 of 500 tokens with 32 rows 57 / 84, 64 rows 94 / 86, 128
// rows 164 / 100.
constexpr int64_t kFewRows = 64;

fp8la_status launch_join(const AttnArgs &a, JoinSide few, JoinSide many, int DP,
                         int64_t rows, cudaStream_t s) {
  few.blocks = static_cast<int32_t>(rows < kRows ? rows : kRows);
  many.blocks = kManyItemRows / kJoinWarps;
  const int blocks = few.ctas * few.blocks + many.ctas * many.blocks;
  if (blocks == 0) return FP8LA_OK;  // no segment has rows, or the call writes nothing
  const int most = many_ctas() * kJoinCtasPerSm - 1;
  const dim3 grid(blocks < most ? blocks : most);
  if (DP == 64) return launch(kv_join_kernel<64>, grid, kJoinThreads, 0, s, a, few, many);
  if (DP == 128) return launch(kv_join_kernel<128>, grid, kJoinThreads, 0, s, a, few, many);
  return launch(kv_join_kernel<256>, grid, kJoinThreads, 0, s, a, few, many);
}

// One pass over all sequences whose rows are at most max_rows (times G): the many-row
// kernel for those with more than kFewRows, the few-row kernel for the others, the join.
// by_many: whether the pass before was the many-row kernel's; becomes whether this one was.
fp8la_status launch_pass(AttnArgs a, const Layout &l, uint8_t *ws, bool f32, int format,
                         int64_t max_rows, bool *by_many, cudaStream_t s) {
  const int DP = padded_dim(a.cache.D);
  auto fits = [](int64_t stride) { return stride >= 0 && stride < (int64_t(1) << 31); };
  const Cache &c = a.cache;
  const bool tc = DP <= 128 && max_rows > kFewRows && fits(c.page_stride / 16) &&
                  fits(c.head_stride / 16) && fits(c.token_stride / 16) &&
                  fits(c.scale_page_stride) && fits(c.scale_head_stride) &&
                  fits(c.scale_token_stride);
  // All rows of a prefix are one sequence, which is all of one kernel's.
  const bool both = !(a.whole && tc);
  // In tiles of either kernel: no more than in tiles of 16 rows against all that the table
  // has room for.
  const auto may_pass = [&](int64_t segments, int64_t tokens) {
    const int64_t rows = static_cast<int64_t>(a.rows.T) * a.G / kRows + segments;
    return rows * c.heads >= INT32_MAX / (tokens / kTile + 1 + kItemCost);
  };
  a.count_other = tc && both && may_pass(a.rows.S, a.rows.capacity);
  a.count_prefix = may_pass(1, a.prefix_capacity);
  JoinSide few = {}, many = {};
  fp8la_status st = FP8LA_OK;
  auto use = [&](const Part &p, int BM, int ctas) {
    a.part_o = reinterpret_cast<float *>(ws + p.o);
    a.part_lse = reinterpret_cast<float *>(ws + p.lse);
    a.desc = reinterpret_cast<Desc *>(ws + p.desc);
    return JoinSide{a.part_o, a.part_lse, a.desc, BM, ctas, 0};
  };
  if (tc) {
    many = use(l.many, kManyItemRows, many_ctas());
    a.row_lo = both ? kFewRows + 1 : 0;
    a.row_hi = INT64_MAX;
    st = launch_many(a, f32, format, many.ctas, s);
  }
  if (st == FP8LA_OK && both) {
    few = use(l.few, kRows, few_ctas(f32, DP));
    a.row_lo = 0;
    a.row_hi = tc ? kFewRows : INT64_MAX;
    // After the many-row kernel, whose workspace is another one; or after the join of a
    // prefix by that kernel, which is the only reader of what this one writes.
    a.late = tc || *by_many;
    st = launch_few(a, f32, format, few.ctas, s);
  }
  *by_many = tc;
  return st == FP8LA_OK ? launch_join(a, few, many, DP, max_rows, s) : st;
}

constexpr int64_t kMaxRowHeads = (int64_t(1) << 31) - (int64_t(1) << 20);
constexpr int32_t kMaxHeads = 65536;  // a tile's tokens times a group's heads fit in 32 bits

}  // namespace

}  // namespace kv
}  // namespace fp8la

using namespace fp8la;
using namespace fp8la::kv;

extern "C" {

int64_t fp8_kv_attention_workspace_bytes(int64_t rows, int32_t num_heads, int32_t head_dim,
                                         int32_t prefix) {
  if (rows < 0 || num_heads < 1 || head_dim < 1) return FP8LA_ERR_INVALID_ARG;
  if (head_dim % 16 != 0 || head_dim > kMaxHeadDim || num_heads > kMaxHeads ||
      rows > INT32_MAX || rows * num_heads >= kMaxRowHeads)
    return FP8LA_ERR_UNSUPPORTED;
  return layout_of(rows, num_heads, head_dim, prefix != 0).bytes;
}

fp8la_status fp8_kv_attention(const void *q, int32_t q_dtype, int64_t ld_q, int64_t ld_q_head,
                              int32_t num_heads, int64_t rows, int64_t num_segments,
                              const int32_t *m_offsets, const int32_t *kv_lens,
                              const int32_t *page_table, int64_t ld_table, int64_t max_pages,
                              int64_t max_rows, const int32_t *prefix_table,
                              int64_t prefix_pages, const int32_t *prefix_len,
                              const fp8la_kv_cache *cache, float scale, int32_t causal,
                              uint16_t *out, int64_t ld_out, int64_t ld_out_head, float *lse,
                              int64_t ld_lse, void *workspace, int64_t workspace_bytes,
                              fp8la_stream_t stream) {
  AttnArgs a = {};
  fp8la_status st = check_cache(cache, &a.cache);
  if (st != FP8LA_OK) return st;
  const int H = a.cache.heads, D = a.cache.D;
  if (q_dtype != FP8LA_TYPE_F32 && q_dtype != FP8LA_TYPE_BF16) return FP8LA_ERR_INVALID_ARG;
  const float scale_log2 = scale * kLog2e;
  if (num_heads < 1 || num_heads % H != 0 || max_rows < 0 || prefix_pages < 0 ||
      !(scale_log2 > -INFINITY && scale_log2 < INFINITY))
    return FP8LA_ERR_INVALID_ARG;
  if (num_heads > kMaxHeads || rows > INT32_MAX || rows * num_heads >= kMaxRowHeads)
    return FP8LA_ERR_UNSUPPORTED;
  st = check_rows(a.cache, m_offsets, kv_lens, page_table, ld_table, max_pages, num_segments,
                  rows, &a.rows);
  if (st != FP8LA_OK || rows == 0 || num_segments == 0) return st;
  const int size = q_dtype == FP8LA_TYPE_F32 ? 4 : 2;
  if (!q || !out || !workspace || (prefix_len && !prefix_table && prefix_pages > 0) ||
      (!prefix_len && prefix_pages > 0))
    return FP8LA_ERR_INVALID_ARG;
  if ((rows > 1 && ld_q < 0) || (num_heads > 1 && ld_q_head < 0)) return FP8LA_ERR_INVALID_ARG;
  const int64_t Hq = num_heads;
  if (!((rows == 1 || ld_out >= (Hq - 1) * ld_out_head + D) && (Hq == 1 || ld_out_head >= D)) &&
      !((Hq == 1 || ld_out_head >= (rows - 1) * ld_out + D) && (rows == 1 || ld_out >= D)))
    return FP8LA_ERR_INVALID_ARG;
  if (lse && rows > 1 && ld_lse < Hq) return FP8LA_ERR_INVALID_ARG;
  const bool prefix = prefix_len != nullptr;
  if (workspace_bytes < fp8_kv_attention_workspace_bytes(rows, num_heads, D, prefix))
    return FP8LA_ERR_INVALID_ARG;
  if (!aligned_to(q, size) || !aligned_to(out, 2) || !aligned_to(lse, 4) ||
      !aligned_to(prefix_table, 4) || !aligned_to(prefix_len, 4) || !aligned16(workspace))
    return FP8LA_ERR_ALIGNMENT;
  if (prefix_pages > INT32_MAX) return FP8LA_ERR_UNSUPPORTED;
  if (!device_is_sm10x()) return FP8LA_ERR_UNSUPPORTED;
  a.rows.status = status_word_ptr();
  if (!a.rows.status) return FP8LA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = q_dtype == FP8LA_TYPE_F32;
  const Layout l = layout_of(rows, num_heads, D, prefix);
  uint8_t *ws = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(workspace) + 255) &
                                            ~uintptr_t(255));
  a.q = q;
  a.ldq = rows > 1 ? ld_q : 0;
  a.ldq_head = num_heads > 1 ? ld_q_head : 0;
  a.out = out;
  a.ldo = rows > 1 ? ld_out : 0;
  a.ldo_head = num_heads > 1 ? ld_out_head : 0;
  a.out_vec = aligned16(out) && a.ldo % 8 == 0 && a.ldo_head % 8 == 0;
  a.lse = lse;
  a.ld_lse = rows > 1 ? ld_lse : 0;
  a.Hq = num_heads;
  a.G = num_heads / H;
  a.group = make_divisor(static_cast<uint32_t>(a.G));
  a.causal = causal != 0;
  a.scale_log2 = scale_log2;
  a.max_rows = max_rows;
  bool by_many = false;
  if (prefix) {
    AttnArgs p = a;
    p.whole = m_offsets + num_segments;
    p.rows.S = 1;
    p.rows.lens = prefix_len;
    p.rows.table = prefix_table;
    p.rows.ld_table = prefix_pages;
    const int64_t most = prefix_pages * a.cache.page_size;
    p.rows.capacity = most < kMaxTokens ? most : kMaxTokens;
    p.causal = 0;
    p.raw_o = reinterpret_cast<float *>(ws + l.raw_o);
    p.raw_lse = reinterpret_cast<float *>(ws + l.raw_lse);
    st = launch_pass(p, l, ws, f32, cache->format, rows * a.G, &by_many, s);
    if (st != FP8LA_OK) return st;
    a.pre_o = p.raw_o;
    a.pre_lse = p.raw_lse;
    a.prefix_len = prefix_len;
    a.prefix_many = by_many;
    a.prefix_capacity = p.rows.capacity;
  }
  const int64_t longest = (max_rows < rows ? max_rows : rows) * a.G;
  return launch_pass(a, l, ws, f32, cache->format, longest, &by_many, s);
}

}  // extern "C"

// Low-rank adapters of many requests beside a shared projection, forward and
// backward.
//
// Rows (tokens) come in segments, one per request; segment s uses adapter
// i = adapter_ids[s], a pair of factors A_i [R][K] and B_i [R][N] and a
// factor alpha_i.  For a row x of the segment:
//
//   forward    v  = A_i x,                 out = base + alpha_i v B_i
//   backward   dv = alpha_i B_i dy,        dx  = dx_base + dv A_i
//              dA_i = sum_t dv_t^T x_t,    dB_i = alpha_i sum_t v_t^T dy_t
//
// Both factors are stored with the rank as the slow dimension, so that three
// kernels make up both directions:
//   shrink   V[t][j]  = sum_k X[t][k] P_i[j][k]       (x, A) and (dy, B)
//   expand   Y[t][n]  = base + sum_j V[t][j] P_i[j][n]  (v, B) and (dv, A)
//   outer    G_i[j][n] = sum_t V[t][j] X[t][n]        (dv, x) and (v, dy)
//
// Bound: HBM.  With R between 8 and 128 every element of X, Y or a factor
// meets few FMAs, so the kernels read each operand once, straight from global
// memory into the fragments of mma.sync (m16n8k16), with no shared memory in
// between: a contraction may take its index in any order, so each lane loads
// 16 consecutive elements of a row and calls them its fragment's, and output
// columns are dealt out so that each lane owns 16 consecutive ones.
//
// Precision: products of BF16 operands are exact and sums FP32.  An FP32
// operand (x or dy given as FP32, v and dv always) enters as a sum of BF16
// terms: three (24 significant bits) where the output is FP32, so that it is
// as good as an FP32 product's, two (relative error 2^-17) where it is
// rounded to BF16.  base + delta is added in FP32 and rounded once.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fp8la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSegments = 1024;
constexpr int kMaxRank = 128;
constexpr int kMaxSplitK = 32;

struct Segments {
  const int32_t *offsets;   // [S + 1]
  const int32_t *ids;       // [S], -1: no adapter
  int32_t S, T, n;
  unsigned *status;
};

// ------------------------------------------------------------ small helpers
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ float bf_lo(uint32_t w) {
  return __uint_as_float(w << 16);
}
__device__ __forceinline__ float bf_hi(uint32_t w) {
  return __uint_as_float(w & 0xffff0000u);
}

// (a, b) as NT BF16 pairs whose sum is the pair to 8 NT significant bits.
// A non-finite value is carried by the first term alone.
template <int NT>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&w)[NT]) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    w[t] = pack_bf16(a, b);
    if (t + 1 < NT) {
      a -= bf_lo(w[t]);
      b -= bf_hi(w[t]);
      if (!(fabsf(a) < 3.0e38f)) a = 0.0f;
      if (!(fabsf(b) < 3.0e38f)) b = 0.0f;
    }
  }
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2 E consecutive elements from column c on of a row of `width` elements, as
// E pairs of BF16 in NT terms; zeros outside the row (p null: all zeros).
template <bool F32, int E, int NT>
__device__ __forceinline__ void load_pairs(const void *p, int64_t c, int64_t width,
                                           bool vec, uint32_t (&w)[NT][E]) {
  if (!F32) {
    const uint16_t *q = static_cast<const uint16_t *>(p) + c;
    if (p && vec && c + 2 * E <= width) {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const uint4 v = *(reinterpret_cast<const uint4 *>(q) + i);
        w[0][4 * i] = v.x;
        w[0][4 * i + 1] = v.y;
        w[0][4 * i + 2] = v.z;
        w[0][4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const uint32_t lo = p && c + 2 * i < width ? q[2 * i] : 0;
        const uint32_t hi = p && c + 2 * i + 1 < width ? q[2 * i + 1] : 0;
        w[0][i] = lo | hi << 16;
      }
    }
  } else {
    const float *q = static_cast<const float *>(p) + c;
    float v[2 * E];
    if (p && vec && c + 2 * E <= width) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float4 f = *(reinterpret_cast<const float4 *>(q) + i);
        v[4 * i] = f.x;
        v[4 * i + 1] = f.y;
        v[4 * i + 2] = f.z;
        v[4 * i + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * E; ++i) v[i] = p && c + i < width ? q[i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      uint32_t t[NT];
      split_pair<NT>(v[2 * i], v[2 * i + 1], t);
#pragma unroll
      for (int k = 0; k < NT; ++k) w[k][i] = t[k];
    }
  }
}

// Exclusive prefix sum over the CTA; total in *all.
__device__ __forceinline__ int block_exclusive(int v, int *warp_sums, int *all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int x = warp_sums[w];
    if (w < warp) before += x;
    total += x;
  }
  __syncthreads();
  *all = total;
  return before + s - v;
}

struct Found {
  int id, row0, rows;  // rows 0: no such tile
};

// Row tile `tile` of the segments cut into tiles of up to TM rows, the rows
// after the last segment counting as one more without an adapter.  Offsets
// that decrease, leave 0..T or ids outside -1..n-1 are recorded and no tile
// is found.
__device__ __forceinline__ Found find_tile(const Segments &g, int tile, int TM,
                                           int *warp_sums, Found *slot) {
  constexpr int kPer = (kMaxSegments + 1 + kThreads - 1) / kThreads;
  // Threads share out the segments evenly, so that few need one round.
  const int per = (g.S + 1 + kThreads - 1) / kThreads;
  int lo[kPer], hi[kPer], sum = 0;
  bool bad = false;
  if (threadIdx.x == 0) *slot = {-1, 0, 0};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = threadIdx.x * per + i;
    lo[i] = hi[i] = 0;
    if (i < per && s <= g.S) {
      lo[i] = g.offsets[s];
      hi[i] = s < g.S ? g.offsets[s + 1] : g.T;
      bad |= lo[i] < 0 || hi[i] < lo[i] || hi[i] > g.T || (s == 0 && lo[i] != 0);
      if (s < g.S) bad |= g.ids[s] < -1 || g.ids[s] >= g.n;
      sum += (hi[i] - lo[i] + TM - 1) / TM;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0) atomicOr(g.status, kStatusBadDeviceArg);
    return {-1, 0, 0};
  }
  int all;
  int at = block_exclusive(sum, warp_sums, &all);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = threadIdx.x * per + i;
    if (i < per && s <= g.S) {
      const int tiles = (hi[i] - lo[i] + TM - 1) / TM;
      if (tile >= at && tile < at + tiles) {
        const int r0 = lo[i] + (tile - at) * TM;
        *slot = {s < g.S ? g.ids[s] : -1, r0, min(TM, hi[i] - r0)};
      }
      at += tiles;
    }
  }
  __syncthreads();
  return *slot;
}

// ------------------------------------------------------------------- shrink
struct ShrinkArgs {
  Segments seg;
  const void *X;
  int64_t ldx;
  const uint16_t *P;
  int64_t ldp, stride_p;
  int64_t K;
  int32_t R, Rp;
  int32_t x_vec, p_vec;
  float *part;  // [K splits][T][Rp]
};

// MT row fragments of 16 rows, NJ rank fragments of 8.  The CTA's eight
// warps take 64-wide K blocks in turn and add their sums in a fixed order.
template <bool F32, int MT, int NJ>
__global__ void __launch_bounds__(kThreads)
    lora_shrink_kernel(const ShrinkArgs a) {
  constexpr int TM = 16 * MT;
  constexpr int NT = F32 ? 3 : 1;
  extern __shared__ float red[];  // [kWarps][TM][8 NJ]
  __shared__ int warp_sums[kWarps];
  __shared__ Found slot;
  pdl_wait();
  pdl_launch_dependents();
  const Found f = find_tile(a.seg, blockIdx.y, TM, warp_sums, &slot);
  if (f.rows == 0 || f.id < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int64_t nkb = (a.K + 63) / 64;
  const int64_t kb0 = nkb * blockIdx.x / gridDim.x;
  const int64_t kb1 = nkb * (blockIdx.x + 1) / gridDim.x;
  const uint16_t *P = a.P + f.id * a.stride_p;
  const int xs = F32 ? 4 : 2;
  float acc[MT][NJ][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.0f;
  for (int64_t kb = kb0 + warp; kb < kb1; kb += kWarps) {
    const int64_t k = kb * 64 + 16 * q;
    uint32_t xa[MT][2][NT][8];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * m + 8 * h + g;
        const char *p = static_cast<const char *>(a.X) +
                        (f.row0 + static_cast<int64_t>(r)) * a.ldx * xs;
        load_pairs<F32, 8, NT>(r < f.rows ? p : nullptr, k, a.K, a.x_vec,
                               xa[m][h]);
      }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int r = 8 * j + g;
      uint32_t pb[1][8];
      load_pairs<false, 8, 1>(r < a.R ? P + r * a.ldp : nullptr, k, a.K,
                              a.p_vec, pb);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma16816(acc[m][j], xa[m][0][t][2 * s], xa[m][1][t][2 * s],
                     xa[m][0][t][2 * s + 1], xa[m][1][t][2 * s + 1],
                     pb[0][2 * s], pb[0][2 * s + 1]);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        red[(warp * TM + 16 * m + g + 8 * (c >> 1)) * (8 * NJ) + 8 * j + 2 * q +
            (c & 1)] = acc[m][j][c];
  __syncthreads();
  float *out = a.part + (static_cast<int64_t>(blockIdx.x) * a.seg.T + f.row0) * a.Rp;
  for (int i = threadIdx.x; i < f.rows * a.Rp; i += kThreads) {
    const int r = i / a.Rp, j = i - r * a.Rp;
    float s = 0.0f;
    if (j < 8 * NJ)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += red[(w * TM + r) * (8 * NJ) + j];
    out[static_cast<int64_t>(r) * a.Rp + j] = s;
  }
}

// ------------------------------------------------------------------- expand
struct ExpandArgs {
  Segments seg;
  const float *part;     // [splits][T][Rp]
  int32_t splits, R, Rp;
  const float *alpha;    // [n]
  int32_t scale_v;       // v_out gets alpha v (backward) instead of v
  float *v_out;          // [T][ldv]
  int64_t ldv;
  const uint16_t *P;     // [n][R][ldp]
  int64_t ldp, stride_p;
  int64_t N;
  const uint16_t *base;
  uint16_t *out;
  int64_t ld_base, ld_out;
  int32_t p_vec, base_vec, out_vec;
};

constexpr int kExpandCols = 64 * kWarps;

__device__ __forceinline__ void load_bf16x16(const uint16_t *p, int64_t c,
                                             int64_t width, bool vec,
                                             uint32_t (&w)[8]) {
  uint32_t t[1][8];
  load_pairs<false, 8, 1>(p, c, width, vec, t);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = t[0][i];
}

__device__ __forceinline__ void store_bf16x16(uint16_t *p, int64_t c,
                                              int64_t width, bool vec,
                                              const uint32_t (&w)[8]) {
  if (vec && c + 16 <= width) {
    uint4 *d = reinterpret_cast<uint4 *>(p + c);
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < width)
        p[c + i] = static_cast<uint16_t>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]);
  }
}

// B fragments of one 16-rank block for this lane's share of 64 columns: rows
// 2q, 2q+1, 2q+8, 2q+9 of the block, columns 8g..8g+7; column i of them is
// column g of fragment i.
__device__ __forceinline__ void load_rank_block(const ExpandArgs &a,
                                                const uint16_t *P, int r0, int q,
                                                int64_t col, uint32_t (&b)[8][2]) {
  uint32_t w[4][1][4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int r = r0 + 2 * q + (h & 1) + 8 * (h >> 1);
    load_pairs<false, 4, 1>(r < a.R ? P + r * a.ldp : nullptr, col, a.N, a.p_vec,
                            w[h]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      b[2 * i][h] = __byte_perm(w[2 * h][0][i], w[2 * h + 1][0][i], 0x5410);
      b[2 * i + 1][h] = __byte_perm(w[2 * h][0][i], w[2 * h + 1][0][i], 0x7632);
    }
}

// One warp per 64 columns; KR blocks of 16 ranks; tiles of TM rows.
template <int TM, int KR>
__global__ void __launch_bounds__(kThreads)
    lora_expand_kernel(const ExpandArgs a) {
  constexpr int kLd = 16 * KR + 8;  // padded row of a term, in BF16
  constexpr bool kHold = KR <= 4;   // the factor stays in registers
  __shared__ __align__(16) uint16_t sv[2][TM][kLd];
  __shared__ int warp_sums[kWarps];
  __shared__ Found slot;
  pdl_wait();
  pdl_launch_dependents();
  const Found f = find_tile(a.seg, blockIdx.y, TM, warp_sums, &slot);
  if (f.rows == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kExpandCols + 64 * warp;
  const bool on = f.id >= 0;
  const float alpha = on ? a.alpha[f.id] : 0.0f;
  const uint16_t *P = a.P + (on ? f.id : 0) * a.stride_p;

  // V of the tile: the K splits added in order, alpha applied, as two terms.
  for (int i = threadIdx.x; i < TM * 8 * KR; i += kThreads) {
    const int r = i / (8 * KR), j = 2 * (i - r * 8 * KR);
    float v0 = 0.0f, v1 = 0.0f;
    if (on && r < f.rows && j < a.Rp)
      for (int s = 0; s < a.splits; ++s) {
        const float2 p = *reinterpret_cast<const float2 *>(
            a.part + ((static_cast<int64_t>(s) * a.seg.T + f.row0 + r) * a.Rp + j));
        v0 += p.x;
        v1 += p.y;
      }
    const float w0 = v0 * alpha, w1 = v1 * alpha;
    if (blockIdx.x == 0 && a.v_out && r < f.rows) {
      float *o = a.v_out + (f.row0 + static_cast<int64_t>(r)) * a.ldv;
      if (j < a.R) o[j] = a.scale_v ? w0 : v0;
      if (j + 1 < a.R) o[j + 1] = a.scale_v ? w1 : v1;
    }
    uint32_t t[2];
    split_pair<2>(w0, w1, t);
    *reinterpret_cast<uint32_t *>(&sv[0][r][j]) = t[0];
    *reinterpret_cast<uint32_t *>(&sv[1][r][j]) = t[1];
  }
  uint32_t b[kHold ? KR : 1][8][2];
  if (kHold && on && col < a.N)
#pragma unroll
    for (int k = 0; k < KR; ++k)
      load_rank_block(a, P, 16 * k, q, col + 8 * g, b[kHold ? k : 0]);
  __syncthreads();
  if (col >= a.N) return;
  for (int m = 0; m < TM / 16 && 16 * m < f.rows; ++m) {
    const int64_t c = col + 16 * q;
    uint32_t w[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 16 * m + 8 * h + g;
      load_bf16x16(r < f.rows ? a.base + (f.row0 + static_cast<int64_t>(r)) * a.ld_base
                              : nullptr,
                   c, a.N, a.base_vec, w[h]);
    }
    float acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
    if (on) {
#pragma unroll
      for (int k = 0; k < KR; ++k) {
        if (!kHold) load_rank_block(a, P, 16 * k, q, col + 8 * g, b[0]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int j = 16 * k + 2 * q;
          const uint32_t a0 = *reinterpret_cast<const uint32_t *>(&sv[t][16 * m + g][j]);
          const uint32_t a1 = *reinterpret_cast<const uint32_t *>(&sv[t][16 * m + g + 8][j]);
          const uint32_t a2 = *reinterpret_cast<const uint32_t *>(&sv[t][16 * m + g][j + 8]);
          const uint32_t a3 =
              *reinterpret_cast<const uint32_t *>(&sv[t][16 * m + g + 8][j + 8]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mma16816(acc[i], a0, a1, a2, a3, b[kHold ? k : 0][i][0],
                     b[kHold ? k : 0][i][1]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 16 * m + 8 * h + g;
      if (r >= f.rows) continue;
      if (on) {
        // Fragment i's columns 2q and 2q + 1 are columns i and 8 + i of the
        // lane's 16.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[h][i] = pack_bf16(bf_lo(w[h][i]) + acc[2 * i][2 * h],
                              bf_hi(w[h][i]) + acc[2 * i + 1][2 * h]);
          w[h][4 + i] = pack_bf16(bf_lo(w[h][4 + i]) + acc[2 * i][2 * h + 1],
                                  bf_hi(w[h][4 + i]) + acc[2 * i + 1][2 * h + 1]);
        }
      }
      store_bf16x16(a.out + (f.row0 + static_cast<int64_t>(r)) * a.ld_out, c, a.N,
                    a.out_vec, w[h]);
    }
  }
}

// -------------------------------------------------------------------- outer
struct OuterSide {
  const float *W;       // [T][ldw]
  int64_t ldw;
  const void *X;        // [T][ldx]
  int64_t ldx;
  int64_t N;
  float *G;             // [n][R][N]
  int32_t x_vec, x_f32;
  int32_t use_alpha;
};
struct OuterArgs {
  Segments seg;
  OuterSide side[2];    // dA (dv, x) and dB (v, dy)
  const float *alpha;
  int32_t R, rank_blocks;
};

constexpr int kColWarps = 4;                    // warps side by side
constexpr int kRowWarps = kWarps / kColWarps;   // warps that share out rows
constexpr int kOuterCols = 64 * kColWarps;

// MR fragments of 16 ranks.  A cluster of CTAs shares out the rows of one
// (adapter, 16 MR ranks, 256 columns) and adds its parts in rank order.
template <bool F32, int MR>
__device__ __forceinline__ void outer_body(const OuterArgs &a, const OuterSide &o,
                                           int adapter, int rank0, int64_t col0,
                                           float *red, int *seg_lo, int *seg_hi,
                                           int *seg_step, int *warp_sums) {
  constexpr int XT = F32 ? 3 : 1;           // terms of X
  constexpr int WT = 3;                     // terms of W
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int cw = warp % kColWarps, rw = warp / kColWarps;
  const uint32_t crank = cluster_ctarank();
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));

  // The adapter's segments, in order, with the steps of 16 rows before each.
  constexpr int kPer = kMaxSegments / kThreads;
  const int per = (a.seg.S + kThreads - 1) / kThreads;
  int lo[kPer], hi[kPer], mine = 0, steps = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = threadIdx.x * per + i;
    lo[i] = hi[i] = 0;
    if (i < per && s < a.seg.S) {
      const int l = a.seg.offsets[s], h = a.seg.offsets[s + 1];
      const int id = a.seg.ids[s];
      bad |= l < 0 || h < l || h > a.seg.T || (s == 0 && l != 0) || id < -1 ||
             id >= a.seg.n;
      if (id == adapter && h > l) {
        lo[i] = l;
        hi[i] = h;
        ++mine;
        steps += (h - l + 15) / 16;
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0) atomicOr(a.seg.status, kStatusBadDeviceArg);
    return;  // every CTA of the grid sees the same
  }
  int nseg, nstep;
  int at = block_exclusive(mine, warp_sums, &nseg);
  int st = block_exclusive(steps, warp_sums, &nstep);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (hi[i] > lo[i]) {
      seg_lo[at] = lo[i];
      seg_hi[at] = hi[i];
      seg_step[at] = st;
      ++at;
      st += (hi[i] - lo[i] + 15) / 16;
    }
  __syncthreads();

  float acc[MR][8][4];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.0f;
  const int s0 = static_cast<int>(static_cast<int64_t>(nstep) * crank / csize);
  const int s1 = static_cast<int>(static_cast<int64_t>(nstep) * (crank + 1) / csize);
  const int64_t c = col0 + 64 * cw + 8 * g;
  int at_seg = 0;
  for (int s = s0 + rw; s < s1; s += kRowWarps) {
    while (at_seg + 1 < nseg && seg_step[at_seg + 1] <= s) ++at_seg;
    const int t0 = seg_lo[at_seg] + 16 * (s - seg_step[at_seg]);
    const int t1 = seg_hi[at_seg];
    // X rows 2q, 2q+1, 2q+8, 2q+9 of the step, columns c..c+7.
    uint32_t x[4][XT][4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int t = t0 + 2 * q + (h & 1) + 8 * (h >> 1);
      const char *p = static_cast<const char *>(o.X) +
                      static_cast<int64_t>(t) * o.ldx * (F32 ? 4 : 2);
      load_pairs<F32, 4, XT>(t < t1 ? p : nullptr, c, o.N, o.x_vec, x[h]);
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      // W of the same rows, ranks g and g + 8 of the block.
      uint32_t wa[4][WT];  // A registers 0..3
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int t = t0 + 2 * q + 8 * (h >> 1);
        const int j = rank0 + 16 * m + g + 8 * (h & 1);
        const float *p = o.W + static_cast<int64_t>(t) * o.ldw + j;
        const float w0 = t < t1 && j < a.R ? p[0] : 0.0f;
        const float w1 = t + 1 < t1 && j < a.R ? p[o.ldw] : 0.0f;
        split_pair<WT>(w0, w1, wa[h]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t sel = i & 1 ? 0x7632u : 0x5410u;
#pragma unroll
        for (int tx = 0; tx < XT; ++tx) {
          const uint32_t b0 = __byte_perm(x[0][tx][i >> 1], x[1][tx][i >> 1], sel);
          const uint32_t b1 = __byte_perm(x[2][tx][i >> 1], x[3][tx][i >> 1], sel);
#pragma unroll
          for (int tw = 0; tw < WT; ++tw)
            if (tx + tw < WT)
              mma16816(acc[m][i], wa[0][tw], wa[1][tw], wa[2][tw], wa[3][tw], b0,
                       b1);
        }
      }
    }
  }

  // Sums of the CTA's row warps, then of the cluster's CTAs, in order.
  constexpr int kLd = kOuterCols + 4;
  for (int w = 0; w < kRowWarps; ++w) {
    if (rw == w) {
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // Fragment i's column n is column 8 n + i of the warp's 64.
            float *d = red + (16 * m + g + 8 * (e >> 1)) * kLd + 64 * cw +
                       8 * (2 * q + (e & 1)) + i;
            *d = w == 0 ? acc[m][i][e] : *d + acc[m][i][e];
          }
    }
    __syncthreads();
  }
  cluster_sync_all();
  const float scale = o.use_alpha ? a.alpha[adapter] : 1.0f;
  const uint32_t red_addr = smem_addr(red);
  constexpr int kCells = 16 * MR * kOuterCols;
  for (int i = static_cast<int>(crank) * kThreads + threadIdx.x; i < kCells;
       i += static_cast<int>(csize) * kThreads) {
    const int r = i / kOuterCols, cc = i % kOuterCols;
    if (rank0 + r >= a.R || col0 + cc >= o.N) continue;
    float s = 0.0f;
    for (uint32_t p = 0; p < csize; ++p) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(v)
                   : "r"(mapa_shared(red_addr + 4u * (r * kLd + cc), p)));
      s += v;
    }
    o.G[(static_cast<int64_t>(adapter) * a.R + rank0 + r) * o.N + col0 + cc] =
        s * scale;
  }
  cluster_sync_all();  // no CTA leaves while its parts are read
}

// grid: x = cluster rank, y = column block of either side, z = adapter and
// rank block.
template <int MR>
__global__ void __launch_bounds__(kThreads)
    lora_outer_kernel(const OuterArgs a) {
  extern __shared__ float red[];  // [16 MR][kOuterCols + 4]
  __shared__ int seg_lo[kMaxSegments], seg_hi[kMaxSegments], seg_step[kMaxSegments];
  __shared__ int warp_sums[kWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int blocks0 = static_cast<int>((a.side[0].N + kOuterCols - 1) / kOuterCols);
  const bool second = static_cast<int>(blockIdx.y) >= blocks0;
  const OuterSide &o = a.side[second];
  const int64_t col0 =
      static_cast<int64_t>(blockIdx.y - (second ? blocks0 : 0)) * kOuterCols;
  const int adapter = blockIdx.z / a.rank_blocks;
  const int rank0 = (blockIdx.z % a.rank_blocks) * 16 * MR;
  if (o.x_f32)
    outer_body<true, MR>(a, o, adapter, rank0, col0, red, seg_lo, seg_hi,
                         seg_step, warp_sums);
  else
    outer_body<false, MR>(a, o, adapter, rank0, col0, red, seg_lo, seg_hi,
                          seg_step, warp_sums);
}

// --------------------------------------------------------------------- host
bool vec_ok(const void *p, int64_t ld, int size, int64_t stride = 0) {
  return aligned16(p) && ld * size % 16 == 0 && stride * size % 16 == 0;
}

// Rows of a tile: short segments get the shortest tile, so that one-token
// requests waste least of a fragment.
bool short_segments(int64_t T, int64_t S) { return T <= 16 * S; }

int64_t tile_bound(int64_t T, int64_t S, int64_t TM) {
  const int64_t most = T / TM + S + 1;
  return most < T ? most : T;
}

int shrink_mt(int64_t T, int64_t S, int R) {
  if (short_segments(T, S)) return 1;
  return R <= 32 ? 4 : R <= 64 ? 2 : 1;
}

// K splits of the shrink kernel: about two CTAs for each SM, each with at
// least one 64-wide block per warp.
int shrink_splits(int64_t T, int64_t S, int64_t K, int R) {
  const int64_t tiles = T / (16 * shrink_mt(T, S, R)) + (S < T ? S : T);
  const int64_t want = (304 + tiles - 1) / (tiles > 0 ? tiles : 1);
  const int64_t most = (K + 64 * kWarps - 1) / (64 * kWarps);
  int64_t s = want < most ? want : most;
  if (s > kMaxSplitK) s = kMaxSplitK;
  return s < 1 ? 1 : static_cast<int>(s);
}

template <typename Kern, typename Args>
fp8la_status launch(Kern kern, dim3 grid, size_t smem, int cluster,
                    const Args &a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? FP8LA_OK
                                                          : FP8LA_ERR_CUDA;
}

template <bool F32, int MT, int NJ>
fp8la_status launch_shrink_one(const ShrinkArgs &a, dim3 grid, cudaStream_t s) {
  constexpr int kSmem = kWarps * 16 * MT * 8 * NJ * 4;
  auto kern = lora_shrink_kernel<F32, MT, NJ>;
  constexpr int slot = 16 + (F32 ? 12 : 0) + (NJ == 1 ? 0 : NJ == 2 ? 1 : NJ == 4 ? 2 : NJ == 8 ? 3 : 4) * 2 + (MT > 1 ? 1 : 0);
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  return launch(kern, grid, kSmem, 0, a, s);
}

template <bool F32>
fp8la_status launch_shrink(const ShrinkArgs &a, int mt, int splits, int64_t T,
                           int64_t S, cudaStream_t s) {
  const dim3 grid(splits, static_cast<unsigned>(tile_bound(T, S, 16 * mt)), 1);
  if (a.R <= 8)
    return mt == 1 ? launch_shrink_one<F32, 1, 1>(a, grid, s)
                   : launch_shrink_one<F32, 4, 1>(a, grid, s);
  if (a.R <= 16)
    return mt == 1 ? launch_shrink_one<F32, 1, 2>(a, grid, s)
                   : launch_shrink_one<F32, 4, 2>(a, grid, s);
  if (a.R <= 32)
    return mt == 1 ? launch_shrink_one<F32, 1, 4>(a, grid, s)
                   : launch_shrink_one<F32, 4, 4>(a, grid, s);
  if (a.R <= 64)
    return mt == 1 ? launch_shrink_one<F32, 1, 8>(a, grid, s)
                   : launch_shrink_one<F32, 2, 8>(a, grid, s);
  return launch_shrink_one<F32, 1, 16>(a, grid, s);
}

template <int TM>
fp8la_status launch_expand_tm(const ExpandArgs &a, int64_t T, int64_t S,
                              cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.N + kExpandCols - 1) / kExpandCols),
                  static_cast<unsigned>(tile_bound(T, S, TM)), 1);
  if (a.R <= 16) return launch(lora_expand_kernel<TM, 1>, grid, 0, 0, a, s);
  if (a.R <= 32) return launch(lora_expand_kernel<TM, 2>, grid, 0, 0, a, s);
  if (a.R <= 64) return launch(lora_expand_kernel<TM, 4>, grid, 0, 0, a, s);
  return launch(lora_expand_kernel<TM, 8>, grid, 0, 0, a, s);
}

fp8la_status launch_expand(const ExpandArgs &a, int64_t T, int64_t S,
                           cudaStream_t s) {
  return short_segments(T, S) ? launch_expand_tm<16>(a, T, S, s)
                              : launch_expand_tm<64>(a, T, S, s);
}

template <int MR>
fp8la_status launch_outer(const OuterArgs &a, int cluster, cudaStream_t s) {
  constexpr int kSmem = 16 * MR * (kOuterCols + 4) * 4;
  auto kern = lora_outer_kernel<MR>;
  if (once_per_device(12 + MR, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  const int64_t blocks = (a.side[0].N + kOuterCols - 1) / kOuterCols +
                         (a.side[1].N + kOuterCols - 1) / kOuterCols;
  return launch(kern, dim3(cluster, static_cast<unsigned>(blocks),
                           static_cast<unsigned>(a.seg.n * a.rank_blocks)),
                kSmem, cluster, a, s);
}

constexpr int64_t kMaxWidth = int64_t(1) << 22;  // grid limits

int64_t part_bytes(int64_t T, int64_t S, int64_t width, int R) {
  return (shrink_splits(T, S, width, R) * T * ((R + 15) / 16 * 16) * 4 + 255) /
         256 * 256;
}

fp8la_status check_common(int64_t T, int32_t S, int32_t n, int32_t R, int64_t K,
                          int64_t N) {
  if (T < 0 || S < 0 || n < 1 || R < 1 || K < 1 || N < 1)
    return FP8LA_ERR_INVALID_ARG;
  if (S > kMaxSegments || R > kMaxRank || T > (int64_t(1) << 19) ||
      K > kMaxWidth || N > kMaxWidth || n > 16383)
    return FP8LA_ERR_UNSUPPORTED;
  return FP8LA_OK;
}

// The factors: BF16 [n][R][ld], adapters `stride` elements apart.
fp8la_status check_factor(const uint16_t *p, int64_t ld, int64_t stride,
                          int64_t width, int32_t n, int32_t R) {
  if (!p || ld < width || (n > 1 && stride < R * ld)) return FP8LA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p) % 2 != 0) return FP8LA_ERR_ALIGNMENT;
  return FP8LA_OK;
}

bool aligned_to(const void *p, int size) {
  return reinterpret_cast<uintptr_t>(p) % size == 0;
}

fp8la_status run_shrink(const Segments &seg, const void *X, int32_t dtype,
                        int64_t ldx, const uint16_t *P, int64_t ldp,
                        int64_t stride, int64_t K, int32_t R, float *part,
                        cudaStream_t s) {
  ShrinkArgs a{};
  a.seg = seg;
  a.X = X;
  a.ldx = ldx;
  a.P = P;
  a.ldp = ldp;
  a.stride_p = stride;
  a.K = K;
  a.R = R;
  a.Rp = (R + 15) / 16 * 16;
  a.x_vec = vec_ok(X, ldx, dtype == FP8LA_TYPE_BF16 ? 2 : 4);
  a.p_vec = vec_ok(P, ldp, 2, stride);
  a.part = part;
  const int mt = shrink_mt(seg.T, seg.S, R);
  const int splits = shrink_splits(seg.T, seg.S, K, R);
  return dtype == FP8LA_TYPE_BF16
             ? launch_shrink<false>(a, mt, splits, seg.T, seg.S, s)
             : launch_shrink<true>(a, mt, splits, seg.T, seg.S, s);
}

fp8la_status run_expand(const Segments &seg, const float *part, int splits,
                        int32_t R, const float *alpha, bool scale_v, float *v,
                        int64_t ldv, const uint16_t *P, int64_t ldp,
                        int64_t stride, int64_t N, const uint16_t *base,
                        int64_t ld_base, uint16_t *out, int64_t ld_out,
                        cudaStream_t s) {
  ExpandArgs a{};
  a.seg = seg;
  a.part = part;
  a.splits = splits;
  a.R = R;
  a.Rp = (R + 15) / 16 * 16;
  a.alpha = alpha;
  a.scale_v = scale_v;
  a.v_out = v;
  a.ldv = ldv;
  a.P = P;
  a.ldp = ldp;
  a.stride_p = stride;
  a.N = N;
  a.base = base;
  a.out = out;
  a.ld_base = ld_base;
  a.ld_out = ld_out;
  a.p_vec = vec_ok(P, ldp, 2, stride);
  a.base_vec = vec_ok(base, ld_base, 2);
  a.out_vec = vec_ok(out, ld_out, 2);
  return launch_expand(a, seg.T, seg.S, s);
}

}  // namespace
}  // namespace fp8la

using namespace fp8la;

extern "C" int64_t fp8la_lora_apply_workspace_bytes(int64_t rows, int32_t segments,
                                                    int64_t K, int32_t rank) {
  const fp8la_status st = check_common(rows, segments, 1, rank, K, 1);
  return st != FP8LA_OK ? st : part_bytes(rows, segments, K, rank);
}

extern "C" int64_t fp8la_lora_backward_workspace_bytes(int64_t rows,
                                                       int32_t segments,
                                                       int64_t N, int32_t rank) {
  const fp8la_status st = check_common(rows, segments, 1, rank, 1, N);
  if (st != FP8LA_OK) return st;
  return part_bytes(rows, segments, N, rank) + rows * ((rank + 15) / 16 * 16) * 4;
}

extern "C" fp8la_status fp8la_lora_apply(
    const uint16_t *base, int64_t ld_base, const void *x, int32_t x_dtype,
    int64_t ldx, int64_t rows, const uint16_t *A, int64_t lda, int64_t stride_a,
    const uint16_t *B, int64_t ldb, int64_t stride_b, const float *alpha,
    int32_t num_adapters, int32_t rank, int64_t K, int64_t N,
    int32_t num_segments, const int32_t *m_offsets, const int32_t *adapter_ids,
    uint16_t *out, int64_t ld_out, float *v, int64_t ldv, void *workspace,
    int64_t workspace_bytes, fp8la_stream_t stream) {
  if (x_dtype != FP8LA_TYPE_F32 && x_dtype != FP8LA_TYPE_BF16)
    return FP8LA_ERR_INVALID_ARG;
  fp8la_status st = check_common(rows, num_segments, num_adapters, rank, K, N);
  if (st != FP8LA_OK) return st;
  if (rows == 0) return FP8LA_OK;
  if (!base || !x || !alpha || !m_offsets || (num_segments > 0 && !adapter_ids) ||
      !out || ld_base < N || ldx < K || ld_out < N || (v && ldv < rank))
    return FP8LA_ERR_INVALID_ARG;
  if (!workspace ||
      workspace_bytes < part_bytes(rows, num_segments, K, rank))
    return FP8LA_ERR_INVALID_ARG;
  if ((st = check_factor(A, lda, stride_a, K, num_adapters, rank)) != FP8LA_OK ||
      (st = check_factor(B, ldb, stride_b, N, num_adapters, rank)) != FP8LA_OK)
    return st;
  if (!aligned_to(base, 2) || !aligned_to(out, 2) || !aligned16(workspace) ||
      !aligned_to(x, x_dtype == FP8LA_TYPE_BF16 ? 2 : 4) || !aligned_to(alpha, 4) ||
      !aligned_to(v, 4))
    return FP8LA_ERR_ALIGNMENT;
  if (!device_is_sm10x()) return FP8LA_ERR_UNSUPPORTED;
  Segments seg{m_offsets, adapter_ids, num_segments, static_cast<int32_t>(rows),
               num_adapters, status_word_ptr()};
  if (!seg.status) return FP8LA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float *part = static_cast<float *>(workspace);
  st = run_shrink(seg, x, x_dtype, ldx, A, lda, stride_a, K, rank, part, s);
  if (st == FP8LA_OK)
    st = run_expand(seg, part, shrink_splits(rows, num_segments, K, rank), rank,
                    alpha, false, v, ldv, B, ldb, stride_b, N, base, ld_base, out,
                    ld_out, s);
  return st == FP8LA_OK ? launch_status() : st;
}

extern "C" fp8la_status fp8la_lora_backward(
    const void *dy, int32_t dy_dtype, int64_t ld_dy, const void *x,
    int32_t x_dtype, int64_t ldx, const float *v, int64_t ldv, int64_t rows,
    const uint16_t *A, int64_t lda, int64_t stride_a, const uint16_t *B,
    int64_t ldb, int64_t stride_b, const float *alpha, int32_t num_adapters,
    int32_t rank, int64_t K, int64_t N, int32_t num_segments,
    const int32_t *m_offsets, const int32_t *adapter_ids,
    const uint16_t *dx_base, int64_t ld_dx_base, uint16_t *dx, int64_t ld_dx,
    float *dA, float *dB, void *workspace, int64_t workspace_bytes,
    fp8la_stream_t stream) {
  if ((x_dtype != FP8LA_TYPE_F32 && x_dtype != FP8LA_TYPE_BF16) ||
      (dy_dtype != FP8LA_TYPE_F32 && dy_dtype != FP8LA_TYPE_BF16))
    return FP8LA_ERR_INVALID_ARG;
  fp8la_status st = check_common(rows, num_segments, num_adapters, rank, K, N);
  if (st != FP8LA_OK) return st;
  if (!dA || !dB || !alpha || !m_offsets || (num_segments > 0 && !adapter_ids))
    return FP8LA_ERR_INVALID_ARG;
  const int Rp = (rank + 15) / 16 * 16;
  const int64_t part = part_bytes(rows, num_segments, N, rank);
  if (rows > 0) {
    if (!dy || !x || !v || !dx_base || !dx || ld_dy < N || ldx < K || ldv < rank ||
        ld_dx_base < K || ld_dx < K || !workspace ||
        workspace_bytes < part + rows * Rp * 4)
      return FP8LA_ERR_INVALID_ARG;
  }
  if ((st = check_factor(A, lda, stride_a, K, num_adapters, rank)) != FP8LA_OK ||
      (st = check_factor(B, ldb, stride_b, N, num_adapters, rank)) != FP8LA_OK)
    return st;
  if (!aligned_to(dy, dy_dtype == FP8LA_TYPE_BF16 ? 2 : 4) ||
      !aligned_to(x, x_dtype == FP8LA_TYPE_BF16 ? 2 : 4) || !aligned_to(v, 4) ||
      !aligned_to(alpha, 4) || !aligned_to(dA, 4) || !aligned_to(dB, 4) ||
      !aligned_to(dx_base, 2) || !aligned_to(dx, 2) || !aligned16(workspace))
    return FP8LA_ERR_ALIGNMENT;
  if (!device_is_sm10x()) return FP8LA_ERR_UNSUPPORTED;
  Segments seg{m_offsets, adapter_ids, num_segments, static_cast<int32_t>(rows),
               num_adapters, status_word_ptr()};
  if (!seg.status) return FP8LA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float *parts = static_cast<float *>(workspace);
  float *dv = reinterpret_cast<float *>(static_cast<char *>(workspace) + part);
  if (rows > 0) {
    st = run_shrink(seg, dy, dy_dtype, ld_dy, B, ldb, stride_b, N, rank, parts, s);
    if (st == FP8LA_OK)
      st = run_expand(seg, parts, shrink_splits(rows, num_segments, N, rank), rank,
                      alpha, true, dv, Rp, A, lda, stride_a, K, dx_base,
                      ld_dx_base, dx, ld_dx, s);
    if (st != FP8LA_OK) return st;
  }
  OuterArgs o{};
  o.seg = seg;
  o.side[0] = {dv, Rp, x, ldx, K, dA, vec_ok(x, ldx, x_dtype == FP8LA_TYPE_BF16 ? 2 : 4),
               x_dtype == FP8LA_TYPE_F32, 0};
  o.side[1] = {v, ldv, dy, ld_dy, N, dB,
               vec_ok(dy, ld_dy, dy_dtype == FP8LA_TYPE_BF16 ? 2 : 4),
               dy_dtype == FP8LA_TYPE_F32, 1};
  o.alpha = alpha;
  o.R = rank;
  const int mr = rank <= 16 ? 1 : 2;
  o.rank_blocks = (rank + 16 * mr - 1) / (16 * mr);
  // CTAs that share out an adapter's rows: 32 rows or more for each of a
  // CTA's row warps.
  int cluster = 1;
  while (cluster < 8 && rows / num_adapters >= 128 * cluster) cluster *= 2;
  st = mr == 1 ? launch_outer<1>(o, cluster, s) : launch_outer<2>(o, cluster, s);
  return st == FP8LA_OK ? launch_status() : st;
}

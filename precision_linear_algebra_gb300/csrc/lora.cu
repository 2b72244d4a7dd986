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
//   shrink   V[t][j]  = sum_k X[t][k] P_i[j][k]         (x, A) and (dy, B)
//   expand   Y[t][n]  = base + sum_j V[t][j] P_i[j][n]  (v, B) and (dv, A)
//   outer    G_i[j][n] = sum_t V[t][j] X[t][n]          (dv, x) and (v, dy)
//
// Bound: HBM.  With R between 8 and 128 every element of X or Y meets few
// FMAs; X and Y are read and written once, and the factors, V and the sums
// are small enough to stay on the chip.  The products are mma.sync m16n8k16
// with fragments from shared memory, filled by cp.async several stages ahead
// (shrink, outer).  In expand a warp keeps its 32 columns of the factor in
// registers and streams rows past them, V from shared memory and base through a
// ring of its own; output columns are dealt out so that each lane owns 8
// consecutive ones.  Sums over a long
// axis (K in shrink, rows in outer) are shared out over a cluster of CTAs and
// added through distributed shared memory in rank order.
//
// Precision: products of BF16 operands are exact and sums FP32.  An FP32
// operand (x or dy given as FP32, v and dv always) enters as a sum of BF16
// terms: three (24 significant bits) where the output is FP32, so that it is
// as good as an FP32 product's, two (relative error 2^-17) where it is
// rounded to BF16.  base is a term of that FP32 sum, which is rounded once.
// The tensor cores cut off a little of a running sum with each addition, always
// towards zero, so V's and the gradients' sums are made of short ones that are
// added with rounding, here of 16 products and in lora_tma.cu of 16 steps:
// whatever the length, they stay as good as an FP32 product's.
//
// Measured on the stream: forward 9.8 us for 8 rows of their own, rank 16, 4096
// -> 4096 (the call's host side takes longer).  The outer sums of FP32 rows
// cost six MMAs a step here: 4096 rows, rank 32, 8192 -> 8192, 221 us backward
// (413 MB, 1.9 TB/s).  BF16 rows at odd addresses are copied element by element:
// 3000 rows, rank 48, 6099 -> 4103, 177 us forward, 87 at even ones.
#include <cuda_bf16.h>

#include "lora.cuh"

namespace fp8la {
namespace {

using namespace lora;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Rows of a matrix are read in units of 16, 8, 4 or 2 bytes, as its address and
// strides allow.
//
// 2 E consecutive BF16 from column c on of a row of `width`, as E pairs; zeros
// outside the row (p null: all zeros).
template <int E>
__device__ __forceinline__ void load_pairs(const uint16_t *p, int64_t c,
                                           int64_t width, int unit,
                                           uint32_t (&w)[E]) {
  const uint16_t *q = p + c;
  if (p && unit == 16 && c + 2 * E <= width) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const uint4 v = *(reinterpret_cast<const uint4 *>(q) + i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else if (E == 2 && p && unit == 8 && c + 2 * E <= width) {
    const uint2 v = *reinterpret_cast<const uint2 *>(q);
    w[0] = v.x;
    w[1] = v.y;
  } else if (p && unit >= 4 && c + 2 * E <= width) {
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] = *(reinterpret_cast<const uint32_t *>(q) + i);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const uint32_t lo = p && c + 2 * i < width ? q[2 * i] : 0;
      const uint32_t hi = p && c + 2 * i + 1 < width ? q[2 * i + 1] : 0;
      w[i] = lo | hi << 16;
    }
  }
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr));
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Copies the U-byte units of `rows` rows of COLS elements of SIZE bytes, see
// copy_tile.
template <int U, int COLS, int SIZE, int LD>
__device__ __forceinline__ void copy_units(uint32_t dst, const char *src, int64_t ld,
                                           int rows, int valid, int64_t c,
                                           int64_t width) {
  constexpr int kUnits = COLS * SIZE / U;
  constexpr int kPer = U / SIZE;
#pragma unroll 4
  for (int i = threadIdx.x; i < rows * kUnits; i += kThreads) {
    const int r = i / kUnits, u = i % kUnits;
    const int64_t cc = c + u * kPer;
    const int n = r < valid && cc < width
                      ? static_cast<int>(min(static_cast<int64_t>(kPer), width - cc)) : 0;
    const char *p = src + (n > 0 ? (r * ld + cc) * SIZE : 0);
    const uint32_t d = dst + r * LD + u * U;
    if (U == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(p),
                   "r"(n * SIZE)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(d), "l"(p),
                   "r"(n * SIZE), "n"(U)
                   : "memory");
  }
}

// Copies `rows` rows of COLS elements of SIZE bytes, from column c of a matrix
// with `width` columns on, to shared memory (rows LD bytes apart), zeros where
// the matrix has no element or r >= valid.  Asynchronous, but for BF16 rows at
// odd addresses, which go through registers, element by element.
template <int COLS, int SIZE, int LD>
__device__ __forceinline__ void copy_tile(uint32_t dst, const char *src, int64_t ld,
                                          int rows, int valid, int64_t c,
                                          int64_t width, int unit) {
  if (unit == 16) {
    copy_units<16, COLS, SIZE, LD>(dst, src, ld, rows, valid, c, width);
  } else if (unit == 8) {
    copy_units<8, COLS, SIZE, LD>(dst, src, ld, rows, valid, c, width);
  } else if (SIZE == 4 || unit == 4) {
    copy_units<4, COLS, SIZE, LD>(dst, src, ld, rows, valid, c, width);
  } else {
    // Neighbouring lanes take neighbouring pairs.
    constexpr int kPairs = COLS / 2;
#pragma unroll 8
    for (int i = threadIdx.x; i < rows * kPairs; i += kThreads) {
      const int r = i / kPairs, u = i % kPairs;
      const int64_t cc = c + 2 * u;
      const uint16_t *p = reinterpret_cast<const uint16_t *>(src) + r * ld + cc;
      const uint32_t lo = r < valid && cc < width ? p[0] : 0;
      const uint32_t hi = r < valid && cc + 1 < width ? p[1] : 0;
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + r * LD + u * 4),
                   "r"(lo | hi << 16)
                   : "memory");
    }
  }
}

// MW groups of warps share out the rows (MF fragments of 16 each), KW = 8 / MW
// the K of a stage; NJ rank fragments of 8 (even where more than one).
template <bool F32, int MW, int MF, int NJ>
struct ShrinkCfg {
  static constexpr int TM = 16 * MW * MF;
  static constexpr int KW = kWarps / MW;
  static constexpr int KS = F32 && KW < 8 ? 64 : 128;  // K of a stage
  static constexpr int kSteps = KS / 16;               // MMA steps of a stage
  static constexpr int RP = 8 * (NJ == 1 ? 2 : NJ);    // ranks in shared memory
  // Padded rows: fragment loads touch every bank once.
  static constexpr int kLdX = KS * (F32 ? 4 : 2) + (F32 ? 32 : 16);
  static constexpr int kLdP = KS * 2 + 16;
  static constexpr int kX = TM * kLdX;
  static constexpr int kStage = kX + RP * kLdP;
  static constexpr int STAGES = kStage * 4 <= 216 * 1024 ? 4 : 3;
  static constexpr int kRing = STAGES * kStage;
  static constexpr int kLdR = 8 * NJ + 2;              // of the sums, in floats
  static constexpr int kRed = KW * TM * kLdR * 4;
  static constexpr int kSmem = kRing > kRed ? kRing : kRed;
  static_assert(kSmem <= 226 * 1024, "shared memory");
  static_assert(kSteps % KW == 0, "every K group has steps");
};

// grid: x = rank in the cluster (K split), y = row tile.
template <bool F32, int MW, int MF, int NJ>
__global__ void __launch_bounds__(kThreads)
    lora_shrink_kernel(const ShrinkArgs a) {
  using C = ShrinkCfg<F32, MW, MF, NJ>;
  constexpr int NT = F32 ? 3 : 1;
  extern __shared__ __align__(16) char smem[];
  __shared__ int warp_sums[kWarps];
  __shared__ Found slot;
  pdl_wait();
  pdl_launch_dependents();
  const Found f = find_tile<kThreads>(a.seg, blockIdx.y, C::TM, warp_sums, &slot);
  if (f.rows == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();
  if (f.id < 0) {  // rows without an adapter
    if (crank == 0)
      for (int i = threadIdx.x; i < f.rows * a.R; i += kThreads)
        a.V[(f.row0 + static_cast<int64_t>(i / a.R)) * a.ldv + i % a.R] = 0.0f;
    return;
  }
  const int g = lane >> 2, q = lane & 3;
  const int mw = warp % MW, kw = warp / MW;
  const int64_t nst = (a.K + C::KS - 1) / C::KS;
  const int s0 = static_cast<int>(nst * crank / csize);
  const int s1 = static_cast<int>(nst * (crank + 1) / csize);
  constexpr int kSize = F32 ? 4 : 2;
  const char *X = static_cast<const char *>(a.X) + f.row0 * a.ldx * kSize;
  const char *P = reinterpret_cast<const char *>(a.P + f.id * a.stride_p);
  const uint32_t base = smem_addr(smem);
  // Rows of fragments that hold no row of the tile are not loaded.
  const int xrows = min(C::TM, (f.rows + 15) / 16 * 16);
  auto fill = [&](int s) {
    if (s < s1) {
      const uint32_t d = base + (s - s0) % C::STAGES * C::kStage;
      const int64_t k = static_cast<int64_t>(s) * C::KS;
      copy_tile<C::KS, kSize, C::kLdX>(d, X, a.ldx, xrows, f.rows, k, a.K, a.x_unit);
      copy_tile<C::KS, 2, C::kLdP>(d + C::kX, P, a.ldp, C::RP, a.R, k, a.K, a.p_unit);
    }
    cp_async_commit();
  };
  float acc[MF][NJ][4];
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.0f;
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) fill(s0 + s);
  for (int s = s0; s < s1; ++s) {
    cp_async_wait<C::STAGES - 2>();
    __syncthreads();
    fill(s + C::STAGES - 1);
    char *sx = smem + (s - s0) % C::STAGES * C::kStage;
    const uint32_t st = smem_addr(sx);
#pragma unroll
    for (int i = 0; i < C::kSteps / C::KW; ++i) {
      const int k = 16 * (kw + i * C::KW);
      uint32_t b[(NJ + 1) / 2][4];
#pragma unroll
      for (int j = 0; j < (NJ + 1) / 2; ++j)
        ldmatrix4(st + C::kX + (16 * j + (lane & 7) + 8 * (lane >> 4)) * C::kLdP +
                      (k + 8 * ((lane >> 3) & 1)) * 2,
                  b[j]);
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        const int r0 = 16 * (mw * MF + m);
        if (r0 >= f.rows) continue;
        uint32_t x[4][NT];
        if (F32) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float2 v = *reinterpret_cast<const float2 *>(
                sx + (r0 + g + 8 * (h & 1)) * C::kLdX + (k + 2 * q + 8 * (h >> 1)) * 4);
            split_pair<NT>(v.x, v.y, x[h]);
          }
        } else {
          uint32_t w[4];
          ldmatrix4(st + (r0 + (lane & 15)) * C::kLdX + (k + 8 * (lane >> 4)) * 2, w);
#pragma unroll
          for (int h = 0; h < 4; ++h) x[h][0] = w[h];
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          // mma.sync cuts off a little of the sum that it adds to, always towards
          // zero: V's relative error after a chain of 256 steps was 2.1e-6, an FP32
          // product's 1e-6 or less.  So each step's 16 products, with FP32 rows all
          // terms of them, the small ones first, are added up apart: 1.3e-7.
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int t = NT - 1; t >= 0; --t)
            mma16816(part, x[0][t], x[1][t], x[2][t], x[3][t], b[j >> 1][2 * (j & 1)],
                     b[j >> 1][2 * (j & 1) + 1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][j][e] += part[e];
        }
      }
    }
  }
  // Sums of the K groups, then of the cluster's CTAs.
  cp_async_wait<0>();
  __syncthreads();
  float *red = reinterpret_cast<float *>(smem);
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int c = 0; c < 4; c += 2)
        *reinterpret_cast<float2 *>(
            red + (kw * C::TM + 16 * (mw * MF + m) + g + 4 * c) * C::kLdR + 8 * j +
            2 * q) = make_float2(acc[m][j][c], acc[m][j][c + 1]);
  __syncthreads();
  const float alpha = a.alpha ? a.alpha[f.id] : 1.0f;
  const int cells = f.rows * a.R;
  if (C::KW > 1 || csize == 1)
    for (int i = threadIdx.x; i < cells; i += kThreads) {
      const int r = i / a.R, j = i - r * a.R;
      float s = red[r * C::kLdR + j];
#pragma unroll
      for (int w = 1; w < C::KW; ++w) s += red[(w * C::TM + r) * C::kLdR + j];
      if (csize == 1)
        a.V[(f.row0 + static_cast<int64_t>(r)) * a.ldv + j] = s * alpha;
      else
        red[r * C::kLdR + j] = s;
    }
  if (csize == 1) return;
  cluster_sync_all();
  for (int i = static_cast<int>(crank) * kThreads + threadIdx.x; i < cells;
       i += static_cast<int>(csize) * kThreads) {
    const int r = i / a.R, j = i - r * a.R;
    a.V[(f.row0 + static_cast<int64_t>(r)) * a.ldv + j] =
        cluster_sum(base + 4u * (r * C::kLdR + j), csize) * alpha;
  }
  cluster_sync_all();  // no CTA leaves while its sums are read
}

// ------------------------------------------------------------------- expand
constexpr int kExpandThreads = 512;
constexpr int kExpandWarps = kExpandThreads / 32;
constexpr int kWarpCols = 32;
constexpr int kExpandCols = kWarpCols * kExpandWarps;

__device__ __forceinline__ void store_bf16x8(uint16_t *p, int64_t c, int64_t width,
                                             int unit, const uint32_t (&w)[4]) {
  if (unit == 16 && c + 8 <= width) {
    *reinterpret_cast<uint4 *>(p + c) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (unit >= 4 && c + 8 <= width) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *(reinterpret_cast<uint32_t *>(p + c) + i) = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < width)
        p[c + i] = static_cast<uint16_t>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]);
  }
}

// B fragments of one 16-rank block for this lane's share of 32 columns: rows
// 2q, 2q+1, 2q+8, 2q+9 of the block, columns 4g..4g+3; column i of them is
// column g of fragment i.
__device__ __forceinline__ void load_rank_block(const ExpandArgs &a,
                                                const uint16_t *P, int r0, int q,
                                                int64_t col, uint32_t (&b)[4][2]) {
  uint32_t w[4][2];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int r = r0 + 2 * q + (h & 1) + 8 * (h >> 1);
    load_pairs<2>(r < a.R ? P + r * a.ldp : nullptr, col, a.N, min(a.p_unit, 8), w[h]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      b[2 * i][h] = __byte_perm(w[2 * h][i], w[2 * h + 1][i], 0x5410);
      b[2 * i + 1][h] = __byte_perm(w[2 * h][i], w[2 * h + 1][i], 0x7632);
    }
}

// One warp per 32 columns, KR blocks of 16 ranks.  A CTA keeps its 512 columns
// and walks down its share of all rows, in chunks of up to CH rows of one
// segment; it fetches the factor's fragments again where the adapter changes.
// While a chunk is multiplied the next one's V is on its way, and each warp
// streams 16-row pieces of base through a ring of its own, RING deep, across
// chunks and segments, with nothing to wait for but its own copies.
constexpr int kPiece = 16 * 2 * kWarpCols;  // bytes: 16 rows of 32 columns

template <int CH, int KR>
struct ExpandCfg {
  static constexpr int RING = CH == 16 ? 2 : 8;
  static constexpr int kLd = 16 * KR + 8;            // padded row of a term, in BF16
  static constexpr int kV = 2 * CH * kLd * 2;        // two terms
  static constexpr int kRingAt = 2 * kV;             // two buffers
  static constexpr int kSegs = kRingAt + kExpandWarps * RING * kPiece;
  static constexpr int kSmem = kSegs + (2 * kMaxSegments + 1) * 4;
  static constexpr int kPairs = (CH * 8 * KR + kExpandThreads - 1) / kExpandThreads;
  static_assert(kV % 16 == 0 && kSmem <= 226 * 1024, "shared memory");
};

template <int CH, int KR>
__global__ void __launch_bounds__(kExpandThreads, 1)
    lora_expand_kernel(const ExpandArgs a) {
  using C = ExpandCfg<CH, KR>;
  extern __shared__ __align__(16) char smem[];
  int *offsets = reinterpret_cast<int *>(smem + C::kSegs);
  int *ids = offsets + a.seg.S + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kExpandCols + kWarpCols * warp;
  const int64_t c = col + 8 * q;
  const int r0 = blockIdx.y * a.rows, r1 = min(a.seg.T, r0 + a.rows);
  pdl_wait();
  pdl_launch_dependents();
  if (!load_segments<kExpandThreads>(a.seg, offsets, ids)) return;
  auto settle = [&](Walk &w) { settle_walk<CH>(w, a.seg.S, offsets, ids, r1); };
  Walk w;
  begin_walk(w, r0, a.seg.S, offsets);
  settle(w);

  const bool live = col < a.N;
  const uint32_t ring = smem_addr(smem) + C::kRingAt + warp * C::RING * kPiece;
  // Rows of 64 bytes; a row's 16-byte units are permuted by its number, so
  // that the eight lanes of a phase meet different banks.
  Walk ahead = w;
  int ahead_p = 0, slot_f = 0;
  auto fetch = [&]() {
    if (a.base_unit >= 4 && live && ahead.row < r1) {
      const int n = ahead.n - ahead_p;
      const uint16_t *src =
          a.base + (ahead.row + static_cast<int64_t>(ahead_p)) * a.ld_base;
      const uint32_t dst = ring + slot_f * kPiece;
      if (a.base_unit == 16) {
        const int u = lane & 3;
        const int64_t left = a.N - (col + 8 * u);
        const int most = left >= 8 ? 16 : left > 0 ? 2 * static_cast<int>(left) : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = (lane >> 2) + 8 * i;
          const int k = r < n ? most : 0;
          const uint16_t *p = k > 0 ? src + r * a.ld_base + col + 8 * u : a.base;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           dst + r * 64 + ((u ^ ((r >> 1) & 3)) << 4)),
                       "l"(p), "r"(k)
                       : "memory");
        }
      } else {
        const int u = lane & 15;
        const int64_t left = a.N - (col + 2 * u);
        const int most = left >= 2 ? 4 : left > 0 ? 2 : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = (lane >> 4) + 2 * i;
          const int k = r < n ? most : 0;
          const uint16_t *p = k > 0 ? src + r * a.ld_base + col + 2 * u : a.base;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                           dst + r * 64 + (((u >> 2) ^ ((r >> 1) & 3)) << 4) +
                           4 * (u & 3)),
                       "l"(p), "r"(k)
                       : "memory");
        }
      }
      ahead_p += 16;
      if (ahead_p >= ahead.n) {
        ahead.row += ahead.n;
        ahead_p = 0;
        if (ahead.row < r1) settle(ahead);
      }
    }
    if (++slot_f == C::RING) slot_f = 0;
    cp_async_commit();
  };
  // Loads only: nothing here waits for them.
  float v[C::kPairs][2], alpha = 1.0f;
  auto load_v = [&](const Walk &w) {
    if (a.alpha && w.row < r1 && w.id >= 0) alpha = __ldg(a.alpha + w.id);
#pragma unroll
    for (int i = 0; i < C::kPairs; ++i) {
      const int e = threadIdx.x + i * kExpandThreads;
      const int r = e / (8 * KR), j = 2 * (e % (8 * KR));
      const bool in = w.row < r1 && w.id >= 0 && r < w.n;
      const float *p = a.V + (w.row + static_cast<int64_t>(r)) * a.ldv + j;
      v[i][0] = in && j < a.R ? __ldcg(p) : 0.0f;
      v[i][1] = in && j + 1 < a.R ? __ldcg(p + 1) : 0.0f;
    }
  };
  auto store_v = [&](int buf) {
    uint16_t *sv = reinterpret_cast<uint16_t *>(smem + buf * C::kV);
#pragma unroll
    for (int i = 0; i < C::kPairs; ++i) {
      const int e = threadIdx.x + i * kExpandThreads;
      const int r = e / (8 * KR), j = 2 * (e % (8 * KR));
      uint32_t t[2];
      split_pair<2>(v[i][0] * alpha, v[i][1] * alpha, t);
      if (r < CH) {
        *reinterpret_cast<uint32_t *>(sv + r * C::kLd + j) = t[0];
        *reinterpret_cast<uint32_t *>(sv + (CH + r) * C::kLd + j) = t[1];
      }
    }
  };

  uint32_t b[KR][4][2];
  int held = -1;
  auto load_factor = [&](int id) {
    if (live && id >= 0 && id != held) {
      held = id;
#pragma unroll
      for (int k = 0; k < KR; ++k)
        load_rank_block(a, a.P + id * a.stride_p, 16 * k, q, col + 4 * g, b[k]);
    }
  };
#pragma unroll
  for (int i = 0; i < C::RING - 1; ++i) fetch();
  load_factor(w.id);
  load_v(w);
  store_v(0);
  int buf = 0, slot = 0;
  while (w.row < r1) {
    __syncthreads();  // V of this chunk is there, the other buffer is free
    Walk next = w;
    next.row += w.n;
    if (next.row < r1) settle(next);
    load_v(next);
    load_factor(w.id);
    const uint32_t sv_lane = smem_addr(smem) + buf * C::kV +
                             ((lane & 15) * C::kLd + 8 * (lane >> 4)) * 2;
    uint16_t *dst = a.out + (w.row + static_cast<int64_t>(g)) * a.ld_out;
    for (int m = 0; m < w.n && live; m += 16, dst += 16 * a.ld_out) {
      cp_async_wait<C::RING - 2>();
      __syncwarp();  // the piece is whole, and the one before it has been read
      // The sums begin with base.  Fragment i's columns 2q and 2q + 1 are
      // columns i and 4 + i of the lane's 8.
      float acc[4][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[4];
        if (a.base_unit >= 4) {
          const uint4 y = *reinterpret_cast<const uint4 *>(
              smem + C::kRingAt + (warp * C::RING + slot) * kPiece + (8 * h + g) * 64 +
              ((q ^ ((g >> 1) & 3)) << 4));
          x[0] = y.x;
          x[1] = y.y;
          x[2] = y.z;
          x[3] = y.w;
        } else {
          const bool in = m + 8 * h + g < w.n;
          load_pairs<4>(in ? a.base + (w.row + m + 8 * h + g) * a.ld_base : nullptr, c,
                        a.N, 2, x);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[2 * i][2 * h] = bf_lo(x[i]);
          acc[2 * i + 1][2 * h] = bf_hi(x[i]);
          acc[2 * i][2 * h + 1] = bf_lo(x[2 + i]);
          acc[2 * i + 1][2 * h + 1] = bf_hi(x[2 + i]);
        }
      }
      fetch();
      if (w.id >= 0) {
#pragma unroll
        for (int k = 0; k < KR; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t f[4];
            ldmatrix4(sv_lane + ((t * CH + m) * C::kLd + 16 * k) * 2, f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma16816(acc[i], f[0], f[1], f[2], f[3], b[k][i][0], b[k][i][1]);
          }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (m + 8 * h + g >= w.n) continue;
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[i] = pack_bf16(acc[2 * i][2 * h], acc[2 * i + 1][2 * h]);
          x[2 + i] = pack_bf16(acc[2 * i][2 * h + 1], acc[2 * i + 1][2 * h + 1]);
        }
        store_bf16x8(dst + 8 * h * a.ld_out, c, a.N, a.out_unit, x);
      }
      if (++slot == C::RING) slot = 0;
    }
    buf ^= 1;
    store_v(buf);
    w = next;
  }
}

// -------------------------------------------------------------------- outer
constexpr int kOuterCols = 32 * kWarps;  // a warp has 32 columns

// MR fragments of 16 ranks.  A stage is up to TS rows of one segment.
template <bool F32, int MR>
struct OuterCfg {
  static constexpr int TS = 32;
  static constexpr int XT = F32 ? 3 : 1;    // terms of X; V has three
  // Padded rows: fragment loads touch every bank once.
  static constexpr int kLdX = kOuterCols * (F32 ? 4 : 2) + 16;
  static constexpr int kX = TS * kLdX;
  static constexpr int STAGES = F32 ? 3 : 4;
  static constexpr int kLdW = 16 * MR + 8;  // row of a term of V, in BF16
  static constexpr int kTerm = TS * kLdW * 2;
  static constexpr int kW = STAGES * kX;    // [2 buffers][3 terms]
  static constexpr int kLdR = kOuterCols + 4;
  static constexpr int kRed = 16 * MR * kLdR * 4;
  static constexpr int kSmem = kW + 6 * kTerm > kRed ? kW + 6 * kTerm : kRed;
  // Words of V (pairs of ranks) that a thread splits for a stage.
  static constexpr int kPairs = TS * 8 * MR / kThreads;
  static_assert(kPairs * kThreads == TS * 8 * MR, "pairs");
  static_assert(kSmem <= 212 * 1024, "shared memory");
};
// CTAs that fit on an SM with either type of X.
template <int MR>
constexpr int kOuterCtas = MR <= 2 ? 2 : 1;

// A cluster of CTAs shares out the rows of one (adapter, 256 columns).
template <bool F32, int MR>
__device__ __forceinline__ void outer_body(const OuterArgs &a, const OuterSide &o,
                                           int adapter, int64_t col0, char *smem,
                                           int *seg_lo, int *seg_hi, int *seg_step,
                                           int *warp_sums) {
  using C = OuterCfg<F32, MR>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();

  // The adapter's segments, in order, with the stages before each.
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
        steps += (h - l + C::TS - 1) / C::TS;
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0) atomicOr(a.seg.status, kStatusBadDeviceArg);
    return;  // every CTA of the grid sees the same
  }
  int nseg, nstep;
  int at = block_exclusive<kThreads>(mine, warp_sums, &nseg);
  int before = block_exclusive<kThreads>(steps, warp_sums, &nstep);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (hi[i] > lo[i]) {
      seg_lo[at] = lo[i];
      seg_hi[at] = hi[i];
      seg_step[at] = before;
      ++at;
      before += (hi[i] - lo[i] + C::TS - 1) / C::TS;
    }
  __syncthreads();

  const int s0 = static_cast<int>(static_cast<int64_t>(nstep) * crank / csize);
  const int s1 = static_cast<int>(static_cast<int64_t>(nstep) * (crank + 1) / csize);
  constexpr int kSize = F32 ? 4 : 2;
  const uint32_t base = smem_addr(smem);
  // First row and number of rows of stage s; `at` follows s upwards.
  auto rows_of = [&](int s, int &at, int &t0) {
    while (at + 1 < nseg && seg_step[at + 1] <= s) ++at;
    t0 = seg_lo[at] + C::TS * (s - seg_step[at]);
    return min(C::TS, seg_hi[at] - t0);
  };
  int at_x = 0, at_w = 0, at_m = 0;
  auto fill = [&](int s) {
    if (s < s1) {
      int t0;
      const int n = rows_of(s, at_x, t0);
      copy_tile<kOuterCols, kSize, C::kLdX>(
          base + (s - s0) % C::STAGES * C::kX,
          static_cast<const char *>(o.X) + t0 * o.ldx * kSize, o.ldx,
          (n + 15) / 16 * 16, n, col0, o.N, o.x_unit);
    }
    cp_async_commit();
  };
  // V of a stage: loaded while the stage before is multiplied, split after it.
  float w[C::kPairs][2];
  auto load_v = [&](int s) {
    int t0 = 0;
    const int n = s < s1 ? rows_of(s, at_w, t0) : 0;
#pragma unroll
    for (int i = 0; i < C::kPairs; ++i) {
      const int e = threadIdx.x + i * kThreads;
      const int r = e / (8 * MR), j = 2 * (e % (8 * MR));
      const float *p = o.W + (t0 + static_cast<int64_t>(r)) * o.ldw + j;
      w[i][0] = r < n && j < a.R ? __ldcg(p) : 0.0f;
      w[i][1] = r < n && j + 1 < a.R ? __ldcg(p + 1) : 0.0f;
    }
  };
  auto store_v = [&](int s) {
    char *d = smem + C::kW + ((s - s0) & 1) * 3 * C::kTerm;
#pragma unroll
    for (int i = 0; i < C::kPairs; ++i) {
      const int e = threadIdx.x + i * kThreads;
      const int r = e / (8 * MR), j = 2 * (e % (8 * MR));
      uint32_t t[3];
      split_pair<3>(w[i][0], w[i][1], t);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint32_t *>(d + k * C::kTerm + (r * C::kLdW + j) * 2) = t[k];
    }
  };
  float acc[MR][4][4];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.0f;
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) fill(s0 + s);
  load_v(s0);
  store_v(s0);
  for (int s = s0; s < s1; ++s) {
    cp_async_wait<C::STAGES - 2>();
    __syncthreads();
    fill(s + C::STAGES - 1);
    load_v(s + 1);
    int t0;
    const int n = rows_of(s, at_m, t0);
    const char *sx = smem + (s - s0) % C::STAGES * C::kX;
    const uint32_t st = smem_addr(sx);
    const uint32_t sw = base + C::kW + ((s - s0) & 1) * 3 * C::kTerm;
#pragma unroll 1
    for (int k = 0; k < n; k += 16) {
      // B: rows k.. of X, the warp's four fragments of 8 columns.
      uint32_t b[C::XT][4][2];
      if (F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float *p = reinterpret_cast<const float *>(
                sx + (k + 2 * q + 8 * h) * C::kLdX + (32 * warp + 8 * i + g) * 4);
            uint32_t t[C::XT];
            split_pair<C::XT>(p[0], p[C::kLdX / 4], t);
#pragma unroll
            for (int x = 0; x < C::XT; ++x) b[x][i][h] = t[x];
          }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t r[4];
          ldmatrix4_trans(st + (k + (lane & 15)) * C::kLdX +
                              (32 * warp + 16 * i + 8 * (lane >> 4)) * 2,
                          r);
          b[0][2 * i][0] = r[0];
          b[0][2 * i][1] = r[1];
          b[0][2 * i + 1][0] = r[2];
          b[0][2 * i + 1][1] = r[3];
        }
      }
#pragma unroll
      for (int m = 0; m < MR; ++m) {
        // mma.sync cuts off a little of the sum that it adds to: over the
        // thousands of rows of an adapter that came to an error of 2e-5.  So
        // 16 rows are added up apart, the small terms first.
        float part[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[i][e] = 0.0f;
#pragma unroll
        for (int t = 2; t >= 0; --t) {
          uint32_t v[4];
          ldmatrix4_trans(sw + t * C::kTerm +
                              ((k + (lane & 7) + 8 * (lane >> 4)) * C::kLdW + 16 * m +
                               8 * ((lane >> 3) & 1)) * 2,
                          v);
#pragma unroll
          for (int x = C::XT - 1; x >= 0; --x)
            if (x + t < 3)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma16816(part[i], v[0], v[1], v[2], v[3], b[x][i][0], b[x][i][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][i][e] += part[i][e];
      }
    }
    if (s + 1 < s1) store_v(s + 1);
  }

  // Sums of the cluster's CTAs, in order.
  cp_async_wait<0>();
  __syncthreads();
  float *red = reinterpret_cast<float *>(smem);
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2)
        *reinterpret_cast<float2 *>(red + (16 * m + g + 4 * e) * C::kLdR + 32 * warp +
                                    8 * i + 2 * q) =
            make_float2(acc[m][i][e], acc[m][i][e + 1]);
  cluster_sync_all();
  // Without rows the gradient is 0 whatever alpha is.
  const float scale = o.use_alpha && nstep > 0 ? a.alpha[adapter] : 1.0f;
  const int cells = a.R * kOuterCols;
  for (int i = static_cast<int>(crank) * kThreads + threadIdx.x; i < cells;
       i += static_cast<int>(csize) * kThreads) {
    const int r = i / kOuterCols, cc = i % kOuterCols;
    if (col0 + cc >= o.N) continue;
    o.G[(static_cast<int64_t>(adapter) * a.R + r) * o.N + col0 + cc] =
        cluster_sum(base + 4u * (r * C::kLdR + cc), csize) * scale;
  }
  cluster_sync_all();  // no CTA leaves while its sums are read
}

// grid: x = cluster rank, y = column block of either side, z = adapter.
template <int MR>
__global__ void __launch_bounds__(kThreads, kOuterCtas<MR>)
    lora_outer_kernel(const OuterArgs a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ int seg_lo[kMaxSegments], seg_hi[kMaxSegments], seg_step[kMaxSegments];
  __shared__ int warp_sums[kWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int blocks0 = static_cast<int>((a.side[0].N + kOuterCols - 1) / kOuterCols);
  const bool second = static_cast<int>(blockIdx.y) >= blocks0;
  const OuterSide &o = a.side[second];
  const int64_t col0 =
      static_cast<int64_t>(blockIdx.y - (second ? blocks0 : 0)) * kOuterCols;
  if (o.x_f32)
    outer_body<true, MR>(a, o, blockIdx.z, col0, smem, seg_lo, seg_hi, seg_step,
                         warp_sums);
  else
    outer_body<false, MR>(a, o, blockIdx.z, col0, smem, seg_lo, seg_hi, seg_step,
                          warp_sums);
}

// --------------------------------------------------------------------- host
// Largest unit, in bytes, that every row of a matrix can be read in.
int unit_of(const void *p, int64_t ld, int size, int64_t stride = 0) {
  const uint64_t all = reinterpret_cast<uintptr_t>(p) |
                       static_cast<uint64_t>(ld * size) |
                       static_cast<uint64_t>(stride * size);
  return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}

template <bool F32, int MW, int MF, int NJ>
fp8la_status launch_shrink_one(const ShrinkArgs &a, int slot, cudaStream_t s) {
  using C = ShrinkCfg<F32, MW, MF, NJ>;
  auto kern = lora_shrink_kernel<F32, MW, MF, NJ>;
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  const int64_t T = a.seg.T, S = a.seg.S;
  // Half of the segments, about, end in a tile of their own.
  const int64_t tiles = T / C::TM + ((S < T ? S : T) + 1) / 2;
  const int64_t slots = sms() * (C::kSmem > 110 * 1024 ? 1 : C::kSmem > 50 * 1024 ? 2 : 4);
  const int cluster = choose_cluster(tiles, (a.K + C::KS - 1) / C::KS, slots, 4);
  return launch(kern,
                dim3(cluster, static_cast<unsigned>(tile_bound(T, S, C::TM)), 1),
                kThreads, C::kSmem, cluster, s, a);
}

template <bool F32, int NJ>
fp8la_status launch_shrink_nj(const ShrinkArgs &a, int slot, cudaStream_t s) {
  // Rows of a tile: 16 for short segments, else 128, or 64 where that leaves
  // too few tiles for the SMs even with K split over whole clusters.
  if (short_segments(a.seg.T, a.seg.S))
    return launch_shrink_one<F32, 1, 1, NJ>(a, slot, s);
  if (a.seg.T < sms() * 128 / kMaxCluster)
    return launch_shrink_one<F32, 4, 1, NJ>(a, slot + 1, s);
  return launch_shrink_one<F32, 4, 2, NJ>(a, slot + 2, s);
}

template <bool F32>
fp8la_status launch_shrink(const ShrinkArgs &a, cudaStream_t s) {
  constexpr int slot = 16 + (F32 ? 15 : 0);
  if (a.R <= 8) return launch_shrink_nj<F32, 1>(a, slot, s);
  if (a.R <= 16) return launch_shrink_nj<F32, 2>(a, slot + 3, s);
  if (a.R <= 32) return launch_shrink_nj<F32, 4>(a, slot + 6, s);
  if (a.R <= 64) return launch_shrink_nj<F32, 8>(a, slot + 9, s);
  return launch_shrink_nj<F32, 16>(a, slot + 12, s);
}

template <int CH, int KR>
fp8la_status launch_expand_one(ExpandArgs a, int slot, cudaStream_t s) {
  using C = ExpandCfg<CH, KR>;
  auto kern = lora_expand_kernel<CH, KR>;
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  // Rows of a CTA: one wave, or a segment or so where those are short, since
  // each brings its own factor.
  const int64_t T = a.seg.T, S = a.seg.S;
  const int64_t blocks = (a.N + kExpandCols - 1) / kExpandCols;
  const int64_t ranges = blocks < sms() ? sms() / blocks : 1;
  int64_t rows = (T + ranges - 1) / ranges;
  if (CH == 16) {
    const int64_t mean = (T + S - 1) / S;
    if (rows > mean) rows = mean;
  } else {
    rows = (rows + 15) / 16 * 16;
  }
  a.rows = static_cast<int32_t>(rows < 1 ? 1 : rows);
  return launch(kern,
                dim3(static_cast<unsigned>(blocks),
                     static_cast<unsigned>((T + a.rows - 1) / a.rows), 1),
                kExpandThreads, C::kSmem, 0, s, a);
}

// CH: rows of a chunk.  V of the largest ranks takes twice the room.
template <int CH>
fp8la_status launch_expand_ch(const ExpandArgs &a, int slot, cudaStream_t s) {
  if (a.R <= 16) return launch_expand_one<CH, 1>(a, slot, s);
  if (a.R <= 32) return launch_expand_one<CH, 2>(a, slot + 1, s);
  if (a.R <= 64) return launch_expand_one<CH, 4>(a, slot + 2, s);
  return launch_expand_one<(CH < 64 ? CH : 64), 8>(a, slot + 3, s);
}

fp8la_status launch_expand(const ExpandArgs &a, cudaStream_t s) {
  // Chunks of 16 rows, a segment to a CTA, spread few short segments over the
  // SMs; with more, loading a factor for each costs more.  Measured, us for a
  // forward pass with chunks of 16 / 128, 4096 -> 4096, rank 16: 8 segments of one
  // row 9.8 / 22.2, 64 of one 24.1 / 40.5, 256 of one 62.5 / 53.2, 1024 of one
  // 220 / 162, 64 of 4 24.3 / 23.1; rank 64: 64 of one 35.6 / 84.9, 256 of one
  // 101.5 / 100.5, 1024 of one 395 / 367, 64 of 16 33.4 / 32.5.
  return a.seg.T < 256 && short_segments(a.seg.T, a.seg.S)
             ? launch_expand_ch<16>(a, 46, s)
             : launch_expand_ch<128>(a, 50, s);
}

template <int MR>
fp8la_status launch_outer(const OuterArgs &a, int slot, cudaStream_t s) {
  constexpr int kSmem = OuterCfg<true, MR>::kSmem > OuterCfg<false, MR>::kSmem
                            ? OuterCfg<true, MR>::kSmem : OuterCfg<false, MR>::kSmem;
  auto kern = lora_outer_kernel<MR>;
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  const int64_t blocks = (a.side[0].N + kOuterCols - 1) / kOuterCols +
                         (a.side[1].N + kOuterCols - 1) / kOuterCols;
  const int cluster = choose_cluster(
      blocks * a.seg.n, (a.seg.T + 32 * a.seg.n - 1) / (32 * a.seg.n),
      sms() * kOuterCtas<MR>, 6);
  return launch(kern, dim3(cluster, static_cast<unsigned>(blocks),
                           static_cast<unsigned>(a.seg.n)),
                kThreads, kSmem, cluster, s, a);
}

// Fewest rows for tcgen05 in shrink and outer: a whole tile.  Below, every call
// takes mma.sync, so that a small call's result does not depend on how its rows
// are aligned.  That has a price: 90 rows in two segments, rank 20, 2048 ->
// 2048, take 15.0 us forward and 27.6 backward, with tcgen05 13.3 and 21.1; 8 rows
// of their own, rank 64, 4096 -> 4096, 15.6 and 46.8 against 12.8 and 34.2.  128
// rows, rank 16, 4096 -> 4096: 12.3 and 24.4 with mma.sync, 10.7 and 18.2 with
// tcgen05.
constexpr int64_t kTmaRows = 128;

constexpr int64_t kMaxWidth = int64_t(1) << 22;  // grid limits

// V (or dv) of every row, FP32.
int64_t v_bytes(int64_t T, int R) { return T * ((R + 3) / 4 * 4) * 4; }

fp8la_status check_common(int64_t T, int32_t S, int32_t n, int32_t R, int64_t K,
                          int64_t N) {
  if (T < 0 || S < 0 || n < 1 || R < 1 || K < 1 || N < 1)
    return FP8LA_ERR_INVALID_ARG;
  if (S > kMaxSegments || R > kMaxRank || T > (int64_t(1) << 19) ||
      K > kMaxWidth || N > kMaxWidth || n > 65535)
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

fp8la_status run_shrink(const Segments &seg, const void *X, int32_t dtype,
                        int64_t ldx, const uint16_t *P, int64_t ldp,
                        int64_t stride, int64_t K, int32_t R, const float *alpha,
                        float *V, int64_t ldv, cudaStream_t s) {
  ShrinkArgs a{};
  a.seg = seg;
  a.X = X;
  a.ldx = ldx;
  a.P = P;
  a.ldp = ldp;
  a.stride_p = stride;
  a.K = K;
  a.R = R;
  a.x_unit = unit_of(X, ldx, dtype == FP8LA_TYPE_BF16 ? 2 : 4);
  a.p_unit = unit_of(P, ldp, 2, stride);
  a.alpha = alpha;
  a.V = V;
  a.ldv = ldv;
  // BF16 rows that TMA can read go to tcgen05, but for short segments of few
  // ranks, whose 128-row tiles are mostly empty.  Measured, us for a forward
  // pass with mma.sync / tcgen05 here, 4096 -> 4096: 256 segments of one row, rank
  // 16: 52.7 / 61.8, rank 32: 78.5 / 76.0, rank 64: 115.2 / 100.5; 1024 of one, rank
  // 16: 162 / 220, rank 32: 258 / 274, rank 64: 394 / 367; 64 of 16, rank 16: 20.9 /
  // 21.5, rank 32: 33.0 / 25.4, rank 64: 47.7 / 32.6.
  if (dtype == FP8LA_TYPE_BF16 && a.x_unit == 16 && a.p_unit == 16 &&
      seg.T >= kTmaRows && (R > 16 || !short_segments(seg.T, seg.S)))
    return launch_shrink_tma(a, s);
  // FP32 rows: splitting a tile costs the same however few of its rows count.
  // mma.sync / tcgen05, 4096 -> 4096: 4 segments, 1024 rows, rank 16: 22.0 / 19.5,
  // rank 64: 39.0 / 24.8, 4096 rows, rank 16: 50.5 / 39.2, rank 64: 82.4 / 46.7;
  // 128 rows, rank 16: 15.6 / 16.5, rank 64: 28.9 / 21.2; rank 64, 64 segments of
  // 16: 54.9 / 57.0, 256 of one: 128 / 187.
  if (dtype == FP8LA_TYPE_F32 && a.x_unit == 16 && a.p_unit == 16 &&
      seg.T >= kTmaRows && !short_segments(seg.T, seg.S))
    return launch_shrink_f32(a, s);
  return dtype == FP8LA_TYPE_BF16 ? launch_shrink<false>(a, s)
                                  : launch_shrink<true>(a, s);
}

fp8la_status run_expand(const Segments &seg, const float *V, int64_t ldv, int32_t R,
                        const float *alpha, const uint16_t *P, int64_t ldp,
                        int64_t stride, int64_t N, const uint16_t *base,
                        int64_t ld_base, uint16_t *out, int64_t ld_out,
                        cudaStream_t s) {
  ExpandArgs a{};
  a.seg = seg;
  a.V = V;
  a.ldv = ldv;
  a.R = R;
  a.alpha = alpha;
  a.P = P;
  a.ldp = ldp;
  a.stride_p = stride;
  a.N = N;
  a.base = base;
  a.out = out;
  a.ld_base = ld_base;
  a.ld_out = ld_out;
  a.p_unit = unit_of(P, ldp, 2, stride);
  a.base_unit = unit_of(base, ld_base, 2);
  a.out_unit = unit_of(out, ld_out, 2);
  a.v_vec = unit_of(V, ldv, 4) == 16;
  // tcgen05 takes 128 rows x 256 columns at a time, wants many such tiles to
  // hide its start, and saves what mma.sync pays for each rank.  Measured, us for
  // a forward pass (K = 1024) with mma.sync / tcgen05 here: rank 16, 4096 x 4096:
  // 23.2 / 25.1, x 10240: 41.9 / 43.4; rank 32, 2048 x 4096: 18.9 / 19.0, x 8192:
  // 27.2 / 25.1, 1024 x 8192: 17.8 / 20.8, 4096 x 4096 in 64 segments: 31.1 /
  // 33.2; rank 64, 2048 x 4096: 25.6 / 22.4, 4096 x 4096: 36.3 / 30.5, 1024 x
  // 8192: 23.7 / 24.3, 4096 x 4096 in 64 segments: 42.9 / 38.5, 2048 x 4096 in 64
  // (K = 4096): 38.9 / 41.9.
  if (a.base_unit == 16 && a.out_unit == 16 && a.p_unit == 16 && R > 16 &&
      R <= 64 && seg.T >= 64 * static_cast<int64_t>(seg.S) && seg.T >= 2048 &&
      seg.T * N >= int64_t(2048) * 4096)
    return launch_expand_tma(a, s);
  return launch_expand(a, s);
}

}  // namespace
}  // namespace fp8la

using namespace fp8la;

extern "C" int64_t fp8la_lora_workspace_bytes(int64_t rows, int32_t rank) {
  const fp8la_status st = check_common(rows, 0, 1, rank, 1, 1);
  return st != FP8LA_OK ? st : v_bytes(rows, rank);
}

extern "C" fp8la_status fp8la_lora_apply(
    const uint16_t *base, int64_t ld_base, const void *x, int32_t x_dtype,
    int64_t ldx, int64_t rows, const uint16_t *A, int64_t lda, int64_t stride_a,
    const uint16_t *B, int64_t ldb, int64_t stride_b, const float *alpha,
    int32_t num_adapters, int32_t rank, int64_t K, int64_t N,
    int32_t num_segments, const int32_t *m_offsets, const int32_t *adapter_ids,
    uint16_t *out, int64_t ld_out, float *v, int64_t ldv,
    fp8la_stream_t stream) {
  if (x_dtype != FP8LA_TYPE_F32 && x_dtype != FP8LA_TYPE_BF16)
    return FP8LA_ERR_INVALID_ARG;
  fp8la_status st = check_common(rows, num_segments, num_adapters, rank, K, N);
  if (st != FP8LA_OK) return st;
  if (rows == 0) return FP8LA_OK;
  if (!base || !x || !alpha || !m_offsets || (num_segments > 0 && !adapter_ids) ||
      !out || !v || ld_base < N || ldx < K || ld_out < N || ldv < rank)
    return FP8LA_ERR_INVALID_ARG;
  if ((st = check_factor(A, lda, stride_a, K, num_adapters, rank)) != FP8LA_OK ||
      (st = check_factor(B, ldb, stride_b, N, num_adapters, rank)) != FP8LA_OK)
    return st;
  if (!aligned_to(base, 2) || !aligned_to(out, 2) ||
      !aligned_to(x, x_dtype == FP8LA_TYPE_BF16 ? 2 : 4) || !aligned_to(alpha, 4) ||
      !aligned_to(v, 4) || !aligned_to(m_offsets, 4) || !aligned_to(adapter_ids, 4))
    return FP8LA_ERR_ALIGNMENT;
  if (!device_is_sm10x()) return FP8LA_ERR_UNSUPPORTED;
  Segments seg{m_offsets, adapter_ids, num_segments, static_cast<int32_t>(rows),
               num_adapters, status_word_ptr()};
  if (!seg.status) return FP8LA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = run_shrink(seg, x, x_dtype, ldx, A, lda, stride_a, K, rank, nullptr, v, ldv, s);
  if (st == FP8LA_OK)
    st = run_expand(seg, v, ldv, rank, alpha, B, ldb, stride_b, N, base, ld_base,
                    out, ld_out, s);
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
  if (rows > 0) {
    if (!dy || !x || !v || !dx_base || !dx || ld_dy < N || ldx < K || ldv < rank ||
        ld_dx_base < K || ld_dx < K || !workspace ||
        workspace_bytes < v_bytes(rows, rank))
      return FP8LA_ERR_INVALID_ARG;
  }
  if ((st = check_factor(A, lda, stride_a, K, num_adapters, rank)) != FP8LA_OK ||
      (st = check_factor(B, ldb, stride_b, N, num_adapters, rank)) != FP8LA_OK)
    return st;
  if (!aligned_to(dy, dy_dtype == FP8LA_TYPE_BF16 ? 2 : 4) ||
      !aligned_to(x, x_dtype == FP8LA_TYPE_BF16 ? 2 : 4) || !aligned_to(v, 4) ||
      !aligned_to(alpha, 4) || !aligned_to(dA, 4) || !aligned_to(dB, 4) ||
      !aligned_to(dx_base, 2) || !aligned_to(dx, 2) || !aligned_to(m_offsets, 4) ||
      !aligned_to(adapter_ids, 4) || !aligned16(workspace))
    return FP8LA_ERR_ALIGNMENT;
  if (!device_is_sm10x()) return FP8LA_ERR_UNSUPPORTED;
  Segments seg{m_offsets, adapter_ids, num_segments, static_cast<int32_t>(rows),
               num_adapters, status_word_ptr()};
  if (!seg.status) return FP8LA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float *dv = static_cast<float *>(workspace);
  const int64_t ld_dv = (rank + 3) / 4 * 4;
  if (rows > 0) {
    st = run_shrink(seg, dy, dy_dtype, ld_dy, B, ldb, stride_b, N, rank, alpha, dv,
                    ld_dv, s);
    if (st == FP8LA_OK)
      st = run_expand(seg, dv, ld_dv, rank, nullptr, A, lda, stride_a, K, dx_base,
                      ld_dx_base, dx, ld_dx, s);
    if (st != FP8LA_OK) return st;
  }
  OuterArgs o{};
  o.seg = seg;
  o.side[0] = {dv, ld_dv, x, ldx, K, dA,
               unit_of(x, ldx, x_dtype == FP8LA_TYPE_BF16 ? 2 : 4),
               x_dtype == FP8LA_TYPE_F32, 0};
  o.side[1] = {v, ldv, dy, ld_dy, N, dB,
               unit_of(dy, ld_dy, dy_dtype == FP8LA_TYPE_BF16 ? 2 : 4),
               dy_dtype == FP8LA_TYPE_F32, 1};
  o.alpha = alpha;
  o.R = rank;
  // BF16 rows that TMA can read.  Measured, us for a backward pass with
  // mma.sync / tcgen05 here, 4096 x 4096, rank 16: 256 segments of one row 129 /
  // 102, 1024 of one 419 / 334, 64 of 16 51.9 / 36.1; rank 64: 256 of one 221 /
  // 206, 64 of 16 89 / 75.
  if (rows >= kTmaRows && !o.side[0].x_f32 && !o.side[1].x_f32 &&
      o.side[0].x_unit == 16 && o.side[1].x_unit == 16) {
    st = launch_outer_tma(o, s);
    return st == FP8LA_OK ? launch_status() : st;
  }
  st = rank <= 16   ? launch_outer<1>(o, 12, s)
       : rank <= 32 ? launch_outer<2>(o, 13, s)
       : rank <= 64 ? launch_outer<4>(o, 14, s)
                    : launch_outer<8>(o, 15, s);
  return st == FP8LA_OK ? launch_status() : st;
}

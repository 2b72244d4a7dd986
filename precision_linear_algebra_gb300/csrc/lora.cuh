// What the adapter kernels share: segments, tiles of their rows, splitting of
// FP32 values into BF16 terms, sums over a cluster, and the launch helpers.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fp8la {
namespace lora {

constexpr int kMaxSegments = 1024;
constexpr int kMaxRank = 128;
constexpr int kMaxCluster = 8;

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

// Sum over the cluster's CTAs, in rank order, of the float at address `addr`
// of each one's shared memory.
__device__ __forceinline__ float cluster_sum(uint32_t addr, uint32_t n) {
  float s = 0.0f;
  for (uint32_t p = 0; p < n; ++p) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                 : "=f"(v)
                 : "r"(mapa_shared(addr, p)));
    s += v;
  }
  return s;
}

// Exclusive prefix sum over the CTA; total in *all.
template <int THREADS>
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
  for (int w = 0; w < THREADS / 32; ++w) {
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
template <int THREADS>
__device__ __forceinline__ Found find_tile(const Segments &g, int tile, int TM,
                                           int *warp_sums, Found *slot) {
  constexpr int kPer = (kMaxSegments + 1 + THREADS - 1) / THREADS;
  // Threads share out the segments evenly, so that few need one round.
  const int per = (g.S + 1 + THREADS - 1) / THREADS;
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
  int at = block_exclusive<THREADS>(sum, warp_sums, &all);
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

struct ShrinkArgs {
  Segments seg;
  const void *X;
  int64_t ldx;
  const uint16_t *P;
  int64_t ldp, stride_p;
  int64_t K;
  int32_t R;
  int32_t x_unit, p_unit;  // bytes that rows can be read in
  const float *alpha;  // null: 1
  float *V;            // [T][ldv]
  int64_t ldv;
};

struct ExpandArgs {
  Segments seg;
  const float *V;        // [T][ldv]
  int64_t ldv;
  int32_t R;
  const float *alpha;    // null: 1
  const uint16_t *P;     // [n][R][ldp]
  int64_t ldp, stride_p;
  int64_t N;
  const uint16_t *base;
  uint16_t *out;
  int64_t ld_base, ld_out;
  int32_t p_unit, base_unit, out_unit;
  int32_t v_vec;         // V's rows can be read in 16-byte units
  int32_t rows;          // of a CTA
};


// Walks down rows: n rows of segment s, which uses adapter id, from `row` on.
struct Walk {
  int row, n, s, id;
};

// Copies the segments to shared memory; false, and recorded, where offsets
// decrease or leave 0..T or ids leave -1..n-1.  Ends with a barrier.
template <int THREADS>
__device__ __forceinline__ bool load_segments(const Segments &g, int *offsets,
                                              int *ids) {
  bool bad = false;
  for (int i = threadIdx.x; i <= g.S; i += THREADS) {
    const int lo = g.offsets[i];
    offsets[i] = lo;
    bad |= lo < 0 || lo > g.T || (i == 0 && lo != 0);
    if (i < g.S) {
      const int id = g.ids[i];
      ids[i] = id;
      bad |= g.offsets[i + 1] < lo || id < -1 || id >= g.n;
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(g.status, kStatusBadDeviceArg);
    return false;
  }
  return true;
}

// A walk from row r0 on (to be settled): the last segment that begins at or
// before it.
__device__ __forceinline__ void begin_walk(Walk &w, int r0, int S, const int *offsets) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= r0) lo = mid;
    else hi = mid - 1;
  }
  w.row = r0;
  w.s = lo;
}

// Finds the segment of w.row (< end) and the rows of it that come next, at
// most CH.  The rows after the last segment count as one more, without an
// adapter.
template <int CH>
__device__ __forceinline__ void settle_walk(Walk &w, int S, const int *offsets,
                                            const int *ids, int end) {
  while (w.s < S && offsets[w.s + 1] <= w.row) ++w.s;
  const int last = min(end, w.s < S ? offsets[w.s + 1] : end);
  w.n = min(CH, last - w.row);
  w.id = w.s < S ? ids[w.s] : -1;
}

struct OuterSide {
  const float *W;       // [T][ldw]
  int64_t ldw;
  const void *X;        // [T][ldx]
  int64_t ldx;
  int64_t N;
  float *G;             // [n][R][N]
  int32_t x_unit, x_f32;
  int32_t use_alpha;
};
struct OuterArgs {
  Segments seg;
  OuterSide side[2];    // dA (dv, x) and dB (v, dy)
  const float *alpha;
  int32_t R;
};

// Rows of a tile: short segments get the shortest tile, so that one-token
// requests waste least of a fragment.
inline bool short_segments(int64_t T, int64_t S) { return T <= 16 * S; }

inline int64_t tile_bound(int64_t T, int64_t S, int64_t TM) {
  const int64_t most = T / TM + S + 1;
  return most < T ? most : T;
}

template <typename Kern, typename... Args>
inline fp8la_status launch(Kern kern, dim3 grid, int threads, size_t smem,
                           int cluster, cudaStream_t s, const Args &...a) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a...) == cudaSuccess ? FP8LA_OK
                                                          : FP8LA_ERR_CUDA;
}

// SMs of the current device (the launch itself fails where there is none).
inline int64_t sms() {
  const int n = sm_count();
  return n > 0 ? n : 1;
}

// CTAs of a cluster that share out a long axis: the least time for `items`
// clusters of `stages` stages each, where a CTA takes about `fixed` stages'
// time to start and to add up, and the SMs hold `slots` CTAs at once (a
// little fewer in large clusters, which have to fit into a GPC).
inline int choose_cluster(int64_t items, int64_t stages, int64_t slots, int fixed) {
  int best = 1;
  double cost = 1e30;
  for (int c = 1; c <= kMaxCluster && (c == 1 || stages >= 2 * c); c *= 2) {
    const int64_t fit = c == 8 ? slots * 7 / 8 : c == 4 ? slots * 15 / 16 : slots;
    const int64_t waves = (items * c + fit - 1) / fit;
    const double t = static_cast<double>(waves) *
                     (static_cast<double>(stages) / c + fixed);
    if (t < cost) {
      cost = t;
      best = c;
    }
  }
  return best;
}

// The same sums for BF16 operands that TMA can read, on tcgen05 (lora_tma.cu).
// V of tiles of 128 rows; base + V P at ranks up to 64; both sides' gradients.
fp8la_status launch_shrink_tma(const ShrinkArgs &a, cudaStream_t s);
fp8la_status launch_shrink_f32(const ShrinkArgs &a, cudaStream_t s);
fp8la_status launch_expand_tma(const ExpandArgs &a, cudaStream_t s);
fp8la_status launch_outer_tma(const OuterArgs &a, cudaStream_t s);

}  // namespace lora
}  // namespace fp8la

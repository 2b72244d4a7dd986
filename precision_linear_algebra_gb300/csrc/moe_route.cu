// Mixture-of-experts router: top-k selection, weights and the row order that
// the expert products need.
//
// For token t with logits z (fp32, or bf16 widened):
//   ids    = the k experts of largest z, larger first, ties to the lowest
//            index; -inf is never chosen (id -1, weight 0), NaN counts as
//            the largest and makes the token's weights NaN
//   weight = exp(z_j - m) / s,  m = max z,  s = the sum of exp(z - m) over
//            the chosen experts (renormalised) or over all of them
// and, where asked for, the stable counting sort of the pairs t * k + slot by
// expert: m_offsets and order, as the grouped calls take them.
//
// One warp holds a token's logits in registers (V per lane), so the
// selection, the maximum and the sum read them once.  A round of the
// selection is two warp reductions: the largest order-preserving integer
// image of a logit, then the lowest index that has it.
//
// The sort is stable without atomics on the positions: each CTA counts the
// pairs of its consecutive tokens per expert, and a second launch turns the
// counts into places.  Up to kClusterTokens tokens a cluster of CTAs, with a
// token for each warp, reads the others' counts from their shared memory: one
// launch and no workspace.
//
// Bound: latency; 8192 x 8 FP32 logits are 0.07 us of memory.  Measured on the
// GPU, with the caches warm: 6.2 us for 1 token, top 8 of 128; sorted, 8.3 us for
// 128 tokens, top 8 of 64 (16.5 in a single CTA, whose warps take the tokens one
// after another) and 14.4 us for 8192 tokens, top 2 of 8, in two launches.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "internal.h"
#include "ptx.cuh"

namespace fp8la {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 16;
// One cluster up to this many tokens.  Above it, two launches on more CTAs.
constexpr int kClusterTokens = 128;
constexpr int kMaxCluster = kClusterTokens / kWarps;
constexpr int kMaxCtas = 256;
constexpr int kMinTokensPerCta = 32;

struct RouteArgs {
  const void *logits;
  int64_t ld;
  int32_t bf16;
  int32_t T, E, k;
  int32_t tokens_per_cta;
  int32_t renorm;
  int32_t *ids;
  float *weights;
  int32_t *m_offsets;  // null: no sort
  int32_t *order;
  int32_t *hist;       // [CTAs][E + 1] (more than one CTA)
};

// Unsigned image of a float whose order is the float's; -0 equals +0.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t u = __float_as_uint(__fadd_rn(z, 0.0f));
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

__device__ __forceinline__ float load_logit(const RouteArgs &a, int64_t i) {
  if (a.bf16)
    return __uint_as_float(
        static_cast<uint32_t>(static_cast<const uint16_t *>(a.logits)[i]) << 16);
  return static_cast<const float *>(a.logits)[i];
}

// Selection and weights of token t by one warp.
template <int V>
__device__ __forceinline__ void route_token(const RouteArgs &a, int t,
                                            int lane) {
  float z[V];
  uint32_t key[V];
  const int64_t row = static_cast<int64_t>(t) * a.ld;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 32 * v;
    z[v] = e < a.E ? load_logit(a, row + e) : -CUDART_INF_F;
    // A NaN counts as the largest, so it is chosen first, becomes m, and
    // makes every weight of the row NaN.
    key[v] = e >= a.E ? kKeyNegInf : z[v] != z[v] ? 0xffffffffu : order_key(z[v]);
  }
  float m = 0.0f, total = 0.0f, mine = 0.0f;
  int my_id = -1;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    best = __reduce_max_sync(0xffffffffu, best);
    if (best <= kKeyNegInf) break;
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
      if (key[v] == best) at = lane + 32 * v;
    at = __reduce_min_sync(0xffffffffu, at);
    const float zj = __uint_as_float((best & 0x80000000u) ? best & 0x7fffffffu
                                                          : ~best);
    if (j == 0) m = zj;
    const float p = expf(zj - m);
    if (a.renorm) total += p;
    if (lane == j) {
      my_id = static_cast<int>(at);
      mine = p;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at == lane + 32u * v) key[v] = kKeyNegInf;
  }
  if (!a.renorm) {
#pragma unroll
    for (int v = 0; v < V; ++v) total += expf(z[v] - m);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      total += __shfl_xor_sync(0xffffffffu, total, d);
  }
  if (lane < a.k) {
    const int64_t o = static_cast<int64_t>(t) * a.k + lane;
    a.ids[o] = my_id;
    a.weights[o] = my_id < 0 ? 0.0f : mine / total;
  }
}

template <int V>
__device__ __forceinline__ void route_tokens(const RouteArgs &a, int t0, int t1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t = t0 + warp; t < t1; t += kWarps) route_token<V>(a, t, lane);
}

__device__ __forceinline__ void route_range(const RouteArgs &a, int t0, int t1) {
  if (a.E <= 32) route_tokens<1>(a, t0, t1);
  else if (a.E <= 64) route_tokens<2>(a, t0, t1);
  else if (a.E <= 128) route_tokens<4>(a, t0, t1);
  else if (a.E <= 256) route_tokens<8>(a, t0, t1);
  else route_tokens<32>(a, t0, t1);
}

// Exclusive prefix sum over the CTA of one value per thread.
__device__ __forceinline__ int block_exclusive(int v, int *warp_sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
  __syncthreads();
  return before + s - v;
}

struct SortSmem {
  int base[kMaxExperts + 1];            // first place of each expert's pairs
  uint16_t by_warp[kWarps][kMaxExperts + 2];  // each warp's pairs per expert
  int warp_sums[kWarps];
};

// Bucket of a pair: its expert, or E (after all experts) for none.
__device__ __forceinline__ int bucket_of(const RouteArgs &a, int64_t pair) {
  const int id = __ldcg(a.ids + pair);
  return id < 0 ? a.E : id;
}

// Places of the pairs [p0, p1), in order, one contiguous part for each warp;
// s.base holds where this CTA's pairs of each bucket begin.
__device__ __forceinline__ void place_pairs(const RouteArgs &a, SortSmem &s,
                                            int64_t p0, int64_t p1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Whole groups of 32 pairs for each warp.
  const int64_t groups = (p1 - p0 + 31) / 32;
  const int64_t lo = min(p1, p0 + (groups * warp / kWarps) * 32);
  const int64_t hi = min(p1, p0 + (groups * (warp + 1) / kWarps) * 32);
  for (int pass = 0; pass < 2; ++pass) {
    for (int64_t g = lo; g < hi; g += 32) {
      const bool in = g + lane < hi;
      const int b = in ? bucket_of(a, g + lane) : kMaxExperts + 1;
      const uint32_t same = __match_any_sync(0xffffffffu, b);
      const int rank = __popc(same & ((1u << lane) - 1u));
      if (pass == 1 && in)
        a.order[s.base[b] + s.by_warp[warp][b] + rank] =
            static_cast<int32_t>(g + lane);
      __syncwarp();
      if (rank == 0 && in)
        s.by_warp[warp][b] =
            static_cast<uint16_t>(s.by_warp[warp][b] + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    if (pass == 0) {
      // Turn the warps' counts into offsets within the CTA's part.
      for (int e = threadIdx.x; e <= a.E; e += kThreads) {
        int run = 0;
        for (int w = 0; w < kWarps; ++w) {
          const int c = s.by_warp[w][e];
          s.by_warp[w][e] = static_cast<uint16_t>(run);
          run += c;
        }
      }
      __syncthreads();
    }
  }
}

// s.base from the buckets' totals and what lies before this CTA's pairs.
// Thread i has the consecutive buckets [i * per, (i + 1) * per).
template <typename Total, typename Before>
__device__ __forceinline__ void bucket_bases(const RouteArgs &a, SortSmem &s,
                                             bool write_offsets, Total total,
                                             Before before) {
  constexpr int kPer = (kMaxExperts + 1 + kThreads - 1) / kThreads;
  int c[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    c[i] = e <= a.E ? total(e) : 0;
    sum += c[i];
  }
  int at = block_exclusive(sum, s.warp_sums);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e <= a.E) {
      s.base[e] = at + before(e);
      if (write_offsets) a.m_offsets[e] = at;  // [E]: all pairs that have one
    }
    at += c[i];
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a) {
  __shared__ SortSmem s;
  __shared__ int count[kMaxExperts + 1];
  const int t0 = blockIdx.x * a.tokens_per_cta;
  const int t1 = min(a.T, t0 + a.tokens_per_cta);
  pdl_launch_dependents();
  route_range(a, t0, t1);
  if (!a.m_offsets) return;
  for (int e = threadIdx.x; e <= a.E; e += kThreads) count[e] = 0;
  __syncthreads();
  const int64_t p0 = static_cast<int64_t>(t0) * a.k;
  const int64_t p1 = static_cast<int64_t>(t1) * a.k;
  // Counts only: their order does not reach the result.
  for (int64_t p = p0 + threadIdx.x; p < p1; p += kThreads)
    atomicAdd(&count[bucket_of(a, p)], 1);
  __syncthreads();
  const uint32_t ranks = cluster_size(), me = cluster_ctarank();
  if (gridDim.x > ranks) {
    for (int e = threadIdx.x; e <= a.E; e += kThreads)
      a.hist[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + e] = count[e];
    return;
  }
  for (int i = threadIdx.x; i < kWarps * (kMaxExperts + 2); i += kThreads)
    (&s.by_warp[0][0])[i] = 0;
  if (ranks == 1) {
    bucket_bases(a, s, true, [&](int e) { return count[e]; },
                 [](int) { return 0; });
    place_pairs(a, s, p0, p1);
    return;
  }
  cluster_sync_all();  // the counts are there
  auto sum = [&](int e, uint32_t n) {
    int v = 0;
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r)
      if (r < n) v += ld_shared_cluster(mapa_shared(smem_addr(&count[e]), r));
    return v;
  };
  bucket_bases(a, s, me == 0, [&](int e) { return sum(e, ranks); },
               [&](int e) { return sum(e, me); });
  place_pairs(a, s, p0, p1);
  cluster_sync_all();  // no CTA leaves while its counts are read
}

// Second launch of a sort over several CTAs: every CTA adds up the counts of
// all CTAs (columns of hist) and places its own pairs.
__global__ void __launch_bounds__(kThreads)
    route_place_kernel(const RouteArgs a, const int ctas) {
  __shared__ SortSmem s;
  __shared__ int total[kMaxExperts + 1], before[kMaxExperts + 1];
  for (int i = threadIdx.x; i < kWarps * (kMaxExperts + 2); i += kThreads)
    (&s.by_warp[0][0])[i] = 0;
  for (int e = threadIdx.x; e <= a.E; e += kThreads) total[e] = before[e] = 0;
  __syncthreads();
  pdl_wait();
  // Rows of hist over the threads, so that few experts still use them all;
  // integer sums, so their order does not matter.
  const int64_t cells = static_cast<int64_t>(ctas) * (a.E + 1);
  for (int64_t i = threadIdx.x; i < cells; i += kThreads) {
    const int c = static_cast<int>(i / (a.E + 1));
    const int e = static_cast<int>(i - static_cast<int64_t>(c) * (a.E + 1));
    const int v = __ldcg(a.hist + i);
    if (v) {
      atomicAdd(&total[e], v);
      if (c < static_cast<int>(blockIdx.x)) atomicAdd(&before[e], v);
    }
  }
  __syncthreads();
  bucket_bases(a, s, blockIdx.x == 0, [&](int e) { return total[e]; },
               [&](int e) { return before[e]; });
  const int t0 = blockIdx.x * a.tokens_per_cta;
  const int t1 = min(a.T, t0 + a.tokens_per_cta);
  place_pairs(a, s, static_cast<int64_t>(t0) * a.k,
              static_cast<int64_t>(t1) * a.k);
}

// Tokens of one CTA: up to kMaxCtas CTAs, so that a CTA of the second launch
// adds up few counts.
int64_t tokens_per_cta(int64_t T) {
  if (T <= kClusterTokens) return kWarps;
  const int64_t per = (T + kMaxCtas - 1) / kMaxCtas;
  return per < kMinTokensPerCta ? kMinTokensPerCta : per;
}

}  // namespace
}  // namespace fp8la

using namespace fp8la;

extern "C" int64_t fp8_moe_route_workspace_bytes(int64_t tokens,
                                                 int32_t num_experts) {
  if (tokens < 0 || num_experts < 1 || num_experts > kMaxExperts)
    return FP8LA_ERR_INVALID_ARG;
  if (tokens <= kClusterTokens) return 0;
  const int64_t per = tokens_per_cta(tokens);
  return (tokens + per - 1) / per * (num_experts + 1) * 4;
}

extern "C" fp8la_status fp8_moe_route(
    const void *logits, int32_t dtype, int64_t tokens, int32_t num_experts,
    int64_t ld, int32_t top_k, int32_t renormalise, int32_t *ids,
    float *weights, int32_t *m_offsets, int32_t *order, void *workspace,
    int64_t workspace_bytes, fp8la_stream_t stream) {
  if (dtype != FP8LA_TYPE_F32 && dtype != FP8LA_TYPE_BF16)
    return FP8LA_ERR_INVALID_ARG;
  if (tokens < 0 || num_experts < 1 || top_k < 1 || top_k > num_experts ||
      ld < num_experts || (order && !m_offsets))
    return FP8LA_ERR_INVALID_ARG;
  if (num_experts > kMaxExperts || top_k > kMaxTopK)
    return FP8LA_ERR_UNSUPPORTED;
  // Token and pair numbers, and those that a loop's last step passes, are 32-bit.
  if (tokens >= ((int64_t(1) << 31) - 65536) / top_k) return FP8LA_ERR_UNSUPPORTED;
  if (tokens > 0 && (!logits || !ids || !weights || (m_offsets && !order)))
    return FP8LA_ERR_INVALID_ARG;
  const bool sort = m_offsets != nullptr;
  const int64_t need = fp8_moe_route_workspace_bytes(tokens, num_experts);
  if (sort && need > 0 && (!workspace || workspace_bytes < need))
    return FP8LA_ERR_INVALID_ARG;
  if (tokens == 0 && !sort) return FP8LA_OK;
  if (!aligned_to(logits, dtype == FP8LA_TYPE_BF16 ? 2 : 4) || !aligned_to(ids, 4) ||
      !aligned_to(weights, 4) || !aligned_to(m_offsets, 4) || !aligned_to(order, 4) ||
      (need > 0 && sort && !aligned_to(workspace, 4)))
    return FP8LA_ERR_ALIGNMENT;
  if (!device_is_sm10x()) return FP8LA_ERR_UNSUPPORTED;
  // A sorting CTA's pairs are counted in 16 bits.
  const int64_t per = tokens_per_cta(tokens);
  if (sort && per * top_k > 65535) return FP8LA_ERR_UNSUPPORTED;
  RouteArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.bf16 = dtype == FP8LA_TYPE_BF16;
  a.T = static_cast<int32_t>(tokens);
  a.E = num_experts;
  a.k = top_k;
  a.tokens_per_cta = static_cast<int32_t>(per);
  a.renorm = renormalise != 0;
  a.ids = ids;
  a.weights = weights;
  a.m_offsets = m_offsets;
  a.order = order;
  a.hist = static_cast<int32_t *>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Without the sort nothing ties the tokens together: one for each warp.
  if (!sort) a.tokens_per_cta = kWarps;
  const int ctas = tokens == 0 ? 1
                               : static_cast<int>((tokens + a.tokens_per_cta - 1) /
                                                  a.tokens_per_cta);
  if (sort && tokens <= kClusterTokens && ctas > 1) {
    unsigned cluster = 2;
    while (cluster < static_cast<unsigned>(ctas)) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(cluster, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_kernel, a) == cudaSuccess
               ? launch_status() : FP8LA_ERR_CUDA;
  }
  route_kernel<<<ctas, kThreads, 0, s>>>(a);
  if (sort && ctas > 1) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, route_place_kernel, a, ctas) != cudaSuccess)
      return FP8LA_ERR_CUDA;
  }
  return launch_status();
}

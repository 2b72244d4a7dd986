// What the key/value cache's kernels share: the cache's layout, the segments of
// a call's rows, where a token lies, and FP8 conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace fp8la {
namespace kv {

constexpr int kMaxSegments = 1024;
constexpr int kMaxHeadDim = 256;
// Tokens of a sequence: a tile and what is requested ahead of it stay below 2^31.
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 4096;

// n / d for 0 <= n < 2^31, by a multiplication: mul = ceil(2^(31 + l) / d) with
// 2^(l-1) < d <= 2^l exceeds 2^(31 + l) / d by less than 2^l / d, so n mul /
// 2^(31 + l) exceeds n / d by less than 1 / d.
struct Divisor {
  uint32_t d, mul, shift;
};
inline Divisor make_divisor(uint32_t d) {
  uint32_t l = 0;
  while ((uint64_t(1) << l) < d) ++l;
  const uint64_t top = uint64_t(1) << (31 + l);
  return {d, static_cast<uint32_t>(d > 1 ? (top + d - 1) / d : 0), l ? l - 1 : 0};
}
__device__ __forceinline__ int divide(int n, const Divisor &v) {
  return v.d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), v.mul) >> v.shift);
}

struct Cache {
  uint8_t *k, *v;            // codes [page][head][place][D]
  float *k_scale, *v_scale;  // [page][head][place]
  int64_t page_stride, head_stride, token_stride;                    // of codes
  int64_t scale_page_stride, scale_head_stride, scale_token_stride;  // of scales
  int32_t num_pages, page_size, heads, D;
  Divisor page;
};

// Segments of the rows of a call: segment s, rows offsets[s] .. offsets[s+1]-1,
// are the last rows of sequence s, which has lens[s] tokens with them, in the
// pages table[s * ld_table ..].
struct Rows {
  const int32_t *offsets, *lens, *table;
  int64_t ld_table, capacity;  // capacity: tokens of a table row
  int32_t S, T;
  unsigned *status;
};

// Copies offsets and lengths to shared memory; false, and recorded, where
// offsets decrease or leave 0..T, or lengths leave 0..capacity or, with `within`,
// are below their segment's rows.  Ends with a barrier.
template <int THREADS>
__device__ __forceinline__ bool load_rows(const Rows &g, bool within, int *offsets,
                                          int *lens) {
  bool bad = false;
  for (int i = threadIdx.x; i <= g.S; i += THREADS) {
    const int lo = g.offsets[i];
    offsets[i] = lo;
    bad |= lo < 0 || lo > g.T || (i == 0 && lo != 0);
    if (i < g.S) {
      const int hi = g.offsets[i + 1], len = g.lens[i];
      lens[i] = len;
      bad |= hi < lo || len < 0 || len > g.capacity ||
             (within && static_cast<int64_t>(len) < static_cast<int64_t>(hi) - lo);
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(g.status, kStatusBadDeviceArg);
    return false;
  }
  return true;
}

// The segment of row t < offsets[S].
__device__ __forceinline__ int segment_of(int t, int S, const int *offsets) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// FP8 formats: 0 = E4M3, 1 = E5M2.
template <int FMT>
struct Format {
  static constexpr float kMax = FMT == 0 ? 448.0f : 57344.0f;
  static constexpr __nv_fp8_interpretation_t kKind = FMT == 0 ? __NV_E4M3 : __NV_E5M2;
  // Codes that are not finite: a NaN for each sign, E5M2's infinities too.
  static __device__ __forceinline__ bool finite(uint32_t code) {
    return FMT == 0 ? (code & 0x7fu) != 0x7fu : (code & 0x7cu) != 0x7cu;
  }
  // The top bit of each of four codes that is not finite.
  static __device__ __forceinline__ uint32_t not_finite4(uint32_t codes) {
    return (FMT == 0 ? (codes & 0x7f7f7f7fu) + 0x01010101u
                     : (codes & 0x7c7c7c7cu) + 0x04040404u) &
           0x80808080u;
  }
  // Takes them out; whether there were any.
  static __device__ __forceinline__ bool clear4(uint32_t &codes) {
    const uint32_t m = not_finite4(codes);
    if (m) codes &= ~((m >> 7) * 255u);
    return m != 0;
  }
};

// Two codes as halves: exact for both formats.
template <int FMT>
__device__ __forceinline__ uint32_t decode2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(codes), Format<FMT>::kKind);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 half2_floats(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The caller's cache, checked.
fp8la_status check_cache(const fp8la_kv_cache *c, Cache *out);
// Segments, checked; a call without rows or segments is left to the caller.
fp8la_status check_rows(const Cache &c, const int32_t *offsets, const int32_t *lens,
                        const int32_t *table, int64_t ld_table, int64_t max_pages,
                        int64_t S, int64_t T, Rows *out);

}  // namespace kv
}  // namespace fp8la

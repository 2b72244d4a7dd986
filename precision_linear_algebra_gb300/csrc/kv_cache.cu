// The key/value cache: rows quantised as they are written, and read back.
//
// A row (token t, head h) of D values has its own scale, as a tensor has one in
// the per-tensor quantiser: amax = max |x|, scale = fp32(amax / fmax), code =
// RNE, saturating, of fp32(x * fp32(fmax / amax)).  Read back: fp32(code * scale).
//
// Bound: HBM, each value once in and once out, and close behind it the instructions
// for each row: BF16 rows write one byte for two read.  D / 8 lanes hold a row, 8 values
// each, so that its amax is a few shuffles and nothing is read twice; a warp takes the
// K and the V of as many heads of a token as it has lanes for, and of up to four times
// as many where there are rows enough, for one look-up of the token's place; the four
// IEEE divisions of a row's K and V are one, each on another lane.  Measured, 65536 rows
// of 8 heads of 128: append of BF16 93 us (4.4 TB/s; 164 with a look-up for each group of
// heads, 118 with four divisions), of FP32 111 us (6.1 TB/s); read as BF16 73 us (5.6
// TB/s), as FP32 139 us (4.9 TB/s).
#include "kv.cuh"

namespace fp8la {
namespace kv {
namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 8;

struct RowSide {
  const void *in;    // append: rows, fp32 or bf16 [T][heads][D]
  void *out;         // read
  int64_t ld, ld_head;
};

struct CopyArgs {
  Rows rows;
  Cache cache;
  RowSide side[2];   // K, V
  int32_t lanes;     // of a row, a power of two
  int32_t blocks;    // groups of heads of a token that a warp has lanes for
  int32_t span;      // of those, in a warp's unit
  int32_t spans;     // units of a token
};

template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const RowSide &s, int64_t at, float (&x)[8]) {
  if (F32) {
    const float *p = static_cast<const float *>(s.in) + at;
    if (VEC) {
      const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
      const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[i];
    }
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(s.in) + at;
    if (VEC) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
    }
  }
}

template <bool F32, bool VEC>
__device__ __forceinline__ void store8(const RowSide &s, int64_t at, const float (&x)[8]) {
  if (F32) {
    float *p = static_cast<float *>(s.out) + at;
    if (VEC) {
      __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
      __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = x[i];
    }
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    uint16_t *p = static_cast<uint16_t *>(s.out) + at;
    if (VEC) {
      __stcs(reinterpret_cast<uint4 *>(p), make_uint4(u[0], u[1], u[2], u[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[2 * i] = static_cast<uint16_t>(u[i]);
        p[2 * i + 1] = static_cast<uint16_t>(u[i] >> 16);
      }
    }
  }
}

// The cache's page and place of row t, or page -1 (recorded) where the table
// names none.
__device__ __forceinline__ int page_of(const CopyArgs &a, int t, const int *offsets,
                                       const int *lens, int *place) {
  const int s = segment_of(t, a.rows.S, offsets);
  const int pos = lens[s] - offsets[s + 1] + t;
  const int p = divide(pos, a.cache.page);
  *place = pos - p * a.cache.page_size;
  const int page = a.rows.table[s * a.rows.ld_table + p];
  if (page >= 0 && page < a.cache.num_pages) return page;
  atomicOr(a.rows.status, kStatusBadDeviceArg);
  return -1;
}

template <bool F32, int FMT, bool VEC, bool APPEND>
__global__ void __launch_bounds__(kThreads, APPEND ? 4 : F32 ? 5 : 8)
    kv_copy_kernel(const CopyArgs a) {
  __shared__ int offsets[kMaxSegments + 1], lens[kMaxSegments + 1];
  pdl_wait();
  pdl_launch_dependents();
  if (!load_rows<kThreads>(a.rows, true, offsets, lens)) return;
  const Cache &c = a.cache;
  const int lane = threadIdx.x & 31, sub = lane & (a.lanes - 1);
  const int per = 32 / a.lanes, d = 8 * sub;
  const uint32_t units = static_cast<uint32_t>(offsets[a.rows.S]) * a.spans;
  const uint32_t step = gridDim.x * (kThreads / 32);
  for (uint32_t u = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units;
       u += step) {
    const int t = u / a.spans, first = (u - t * a.spans) * a.span;
    const int64_t row0 = t * a.side[0].ld + d, row1 = t * a.side[1].ld + d;
    const int last = min(first + a.span, a.blocks) - 1;
    float x[2][8] = {};
    auto load = [&](int block) {
      const int h = block * per + lane / a.lanes;
      if (h >= c.heads || d >= c.D) return;
      load8<F32, VEC>(a.side[0], row0 + h * a.side[0].ld_head, x[0]);
      load8<F32, VEC>(a.side[1], row1 + h * a.side[1].ld_head, x[1]);
    };
    // Rows are on their way while the token's place is looked up.
    if (APPEND) load(first);
    int place;
    const int page = page_of(a, t, offsets, lens, &place);
    const int64_t code0 = page * c.page_stride + place * c.token_stride + d;
    const int64_t scale0 = page * c.scale_page_stride + place * c.scale_token_stride;
#pragma unroll 1
    for (int block = first; block <= last; ++block) {
      const int h = block * per + lane / a.lanes;
      const bool on = h < c.heads && d < c.D;
      const int64_t at0 = row0 + h * a.side[0].ld_head, at1 = row1 + h * a.side[1].ld_head;
      const int64_t code = code0 + h * c.head_stride, scale = scale0 + h * c.scale_head_stride;
      if (APPEND) {
        if (block > first) load(block);
        float m[2];  // fmaxf drops NaN
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          m[i] = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) m[i] = fmaxf(m[i], fabsf(x[i][j]));
        }
        for (int o = a.lanes >> 1; o > 0; o >>= 1) {
#pragma unroll
          for (int i = 0; i < 2; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
        }
        // Four divisions at once, each on another lane of the row: fmax / amax of K and
        // of V, amax / fmax of K and of V.  Rows of 16 have but two lanes.
        constexpr float kMax = Format<FMT>::kMax;
        float up[2], down;
        if (a.lanes >= 4) {
          const float own = sub & 1 ? m[1] : m[0];
          const float q = __fdiv_rn(sub & 2 ? own : kMax, sub & 2 ? kMax : own);
          up[0] = __shfl_sync(0xffffffffu, q, lane & ~3);
          up[1] = __shfl_sync(0xffffffffu, q, lane & ~3 | 1);
          down = q;
        } else {
          up[0] = __fdiv_rn(kMax, m[0]);
          up[1] = __fdiv_rn(kMax, m[1]);
          down = __fdiv_rn(sub ? m[1] : m[0], kMax);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool none = m[i] == 0.0f || !isfinite(up[i]);
          if (none) up[i] = 1.0f;
          uint32_t w[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 8; j += 2)
            w[j >> 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                             make_float2(x[i][j] * up[i], x[i][j + 1] * up[i]), __NV_SATFINITE,
                             Format<FMT>::kKind))
                         << (8 * (j & 3));
          if (on && page >= 0) {
            *reinterpret_cast<uint2 *>((i == 0 ? c.k : c.v) + code) = make_uint2(w[0], w[1]);
            if (sub == (a.lanes >= 4 ? 2 + i : i))
              (i == 0 ? c.k_scale : c.v_scale)[scale] = none ? 1.0f : down;
          }
        }
      } else if (on && page >= 0) {
        const uint2 wk = *reinterpret_cast<const uint2 *>(c.k + code);
        const uint2 wv = *reinterpret_cast<const uint2 *>(c.v + code);
        const float s[2] = {c.k_scale[scale], c.v_scale[scale]};
        const uint32_t w[2][2] = {{wk.x, wk.y}, {wv.x, wv.y}};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = half2_floats(decode2<FMT>((w[i][j >> 1] >> (16 * (j & 1))) & 0xffffu));
            x[i][2 * j] = f.x * s[i];
            x[i][2 * j + 1] = f.y * s[i];
          }
          store8<F32, VEC>(a.side[i], i == 0 ? at0 : at1, x[i]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------- host
template <bool F32, int FMT, bool VEC, bool APPEND>
fp8la_status launch_copy(const CopyArgs &a, cudaStream_t s) {
  const int64_t units = static_cast<int64_t>(a.rows.T) * a.spans;
  const int64_t ctas = (units + kThreads / 32 - 1) / (kThreads / 32);
  const int sms = sm_count();
  const int64_t most = static_cast<int64_t>(sms > 0 ? sms : 1) * kCtasPerSm;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_copy_kernel<F32, FMT, VEC, APPEND>, a) == cudaSuccess
             ? FP8LA_OK
             : FP8LA_ERR_CUDA;
}

template <bool APPEND>
fp8la_status copy(const fp8la_kv_cache *cache, const RowSide &k, const RowSide &v,
                  int32_t dtype, int64_t T, int64_t S, const int32_t *offsets,
                  const int32_t *lens, const int32_t *table, int64_t ld_table,
                  int64_t max_pages, cudaStream_t s) {
  CopyArgs a = {};
  fp8la_status st = check_cache(cache, &a.cache);
  if (st != FP8LA_OK) return st;
  if (dtype != FP8LA_TYPE_F32 && dtype != FP8LA_TYPE_BF16) return FP8LA_ERR_INVALID_ARG;
  st = check_rows(a.cache, offsets, lens, table, ld_table, max_pages, S, T, &a.rows);
  if (st != FP8LA_OK || T == 0 || S == 0) return st;
  const int size = dtype == FP8LA_TYPE_F32 ? 4 : 2;
  a.side[0] = k;
  a.side[1] = v;
  bool vec = true;
  for (const RowSide &r : a.side) {
    const void *p = APPEND ? r.in : r.out;
    const int64_t D = a.cache.D, H = a.cache.heads;
    if (!p || (T > 1 && r.ld < 0) || (H > 1 && r.ld_head < 0)) return FP8LA_ERR_INVALID_ARG;
    // Rows that are written lie apart, tokens or heads outside.
    if (!APPEND && !((T == 1 || r.ld >= (H - 1) * r.ld_head + D) && (H == 1 || r.ld_head >= D)) &&
        !((H == 1 || r.ld_head >= (T - 1) * r.ld + D) && (T == 1 || r.ld >= D)))
      return FP8LA_ERR_INVALID_ARG;
    if (!aligned_to(p, size)) return FP8LA_ERR_ALIGNMENT;
    vec = vec && aligned16(p) && (T == 1 || r.ld * size % 16 == 0) &&
          (a.cache.heads == 1 || r.ld_head * size % 16 == 0);
  }
  int lanes = 2;
  while (lanes * 8 < a.cache.D) lanes *= 2;
  a.lanes = lanes;
  a.blocks = (a.cache.heads + 32 / lanes - 1) / (32 / lanes);
  // One look-up of a token's place for several groups of heads, unless that left SMs
  // without work.
  const int64_t full = static_cast<int64_t>(sm_count()) * kCtasPerSm * (kThreads / 32);
  a.span = T * a.blocks >= 4 * full ? 4 : 1;
  a.spans = (a.blocks + a.span - 1) / a.span;
  if (T * a.blocks >= (int64_t(1) << 31) - (int64_t(1) << 20)) return FP8LA_ERR_UNSUPPORTED;
  if (!device_is_sm10x()) return FP8LA_ERR_UNSUPPORTED;
  a.rows.status = status_word_ptr();
  if (!a.rows.status) return FP8LA_ERR_CUDA;
  const int which = (dtype == FP8LA_TYPE_F32 ? 4 : 0) |
                    (cache->format == FP8LA_FORMAT_E5M2 ? 2 : 0) | (vec ? 1 : 0);
  switch (which) {
    case 0: return launch_copy<false, 0, false, APPEND>(a, s);
    case 1: return launch_copy<false, 0, true, APPEND>(a, s);
    case 2: return launch_copy<false, 1, false, APPEND>(a, s);
    case 3: return launch_copy<false, 1, true, APPEND>(a, s);
    case 4: return launch_copy<true, 0, false, APPEND>(a, s);
    case 5: return launch_copy<true, 0, true, APPEND>(a, s);
    case 6: return launch_copy<true, 1, false, APPEND>(a, s);
    default: return launch_copy<true, 1, true, APPEND>(a, s);
  }
}

}  // namespace

fp8la_status check_cache(const fp8la_kv_cache *c, Cache *out) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return FP8LA_ERR_INVALID_ARG;
  if (c->format != FP8LA_FORMAT_E4M3 && c->format != FP8LA_FORMAT_E5M2)
    return FP8LA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1)
    return FP8LA_ERR_INVALID_ARG;
  if (c->head_dim % 16 != 0 || c->head_dim > kMaxHeadDim || c->kv_heads > 1024 ||
      c->num_pages > INT32_MAX || c->page_size > (1 << 30))
    return FP8LA_ERR_UNSUPPORTED;
  // Strides of dimensions of one element address nothing.
  if ((c->page_size > 1 && c->token_stride < c->head_dim) ||
      (c->kv_heads > 1 && c->head_stride < c->head_dim) ||
      (c->num_pages > 1 && c->page_stride < c->head_dim))
    return FP8LA_ERR_INVALID_ARG;
  if ((c->num_pages > 1 && c->scale_page_stride < 1) ||
      (c->kv_heads > 1 && c->scale_head_stride < 1) ||
      (c->page_size > 1 && c->scale_token_stride < 1))
    return FP8LA_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned_to(c->k_scale, 4) ||
      !aligned_to(c->v_scale, 4) || (c->num_pages > 1 && c->page_stride % 16 != 0) ||
      (c->kv_heads > 1 && c->head_stride % 16 != 0) ||
      (c->page_size > 1 && c->token_stride % 16 != 0))
    return FP8LA_ERR_ALIGNMENT;
  *out = {c->k, c->v, c->k_scale, c->v_scale,
          c->num_pages > 1 ? c->page_stride : 0, c->kv_heads > 1 ? c->head_stride : 0,
          c->page_size > 1 ? c->token_stride : 0,
          c->num_pages > 1 ? c->scale_page_stride : 0,
          c->kv_heads > 1 ? c->scale_head_stride : 0,
          c->page_size > 1 ? c->scale_token_stride : 0,
          static_cast<int32_t>(c->num_pages), c->page_size, c->kv_heads, c->head_dim,
          make_divisor(static_cast<uint32_t>(c->page_size))};
  return FP8LA_OK;
}

fp8la_status check_rows(const Cache &c, const int32_t *offsets, const int32_t *lens,
                        const int32_t *table, int64_t ld_table, int64_t max_pages,
                        int64_t S, int64_t T, Rows *out) {
  if (S < 0 || T < 0 || max_pages < 0 || (S > 1 && ld_table < max_pages))
    return FP8LA_ERR_INVALID_ARG;
  if (S > kMaxSegments || T > INT32_MAX || max_pages > INT32_MAX)
    return FP8LA_ERR_UNSUPPORTED;
  if (S == 0 || T == 0) return FP8LA_OK;
  if (!offsets || !lens || (!table && max_pages > 0)) return FP8LA_ERR_INVALID_ARG;
  if (!aligned_to(offsets, 4) || !aligned_to(lens, 4) || !aligned_to(table, 4))
    return FP8LA_ERR_ALIGNMENT;
  const int64_t most = max_pages * c.page_size;
  *out = {offsets, lens, table, ld_table,
          most < kMaxTokens ? most : kMaxTokens,
          static_cast<int32_t>(S), static_cast<int32_t>(T), nullptr};
  return FP8LA_OK;
}

}  // namespace kv
}  // namespace fp8la

extern "C" {

fp8la_status fp8_kv_append(const void *k, int64_t ld_k, int64_t ld_k_head, const void *v,
                           int64_t ld_v, int64_t ld_v_head, int32_t dtype, int64_t rows,
                           int64_t num_segments, const int32_t *m_offsets,
                           const int32_t *kv_lens, const int32_t *page_table,
                           int64_t ld_table, int64_t max_pages,
                           const fp8la_kv_cache *cache, fp8la_stream_t stream) {
  return fp8la::kv::copy<true>(cache, {k, nullptr, ld_k, ld_k_head},
                               {v, nullptr, ld_v, ld_v_head}, dtype, rows, num_segments,
                               m_offsets, kv_lens, page_table, ld_table, max_pages,
                               reinterpret_cast<cudaStream_t>(stream));
}

fp8la_status fp8_kv_read(void *k, int64_t ld_k, int64_t ld_k_head, void *v, int64_t ld_v,
                         int64_t ld_v_head, int32_t dtype, int64_t rows,
                         int64_t num_segments, const int32_t *m_offsets,
                         const int32_t *kv_lens, const int32_t *page_table,
                         int64_t ld_table, int64_t max_pages, const fp8la_kv_cache *cache,
                         fp8la_stream_t stream) {
  return fp8la::kv::copy<false>(cache, {nullptr, k, ld_k, ld_k_head},
                                {nullptr, v, ld_v, ld_v_head}, dtype, rows, num_segments,
                                m_offsets, kv_lens, page_table, ld_table, max_pages,
                                reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// What the attention kernels share: their arguments, how the work is shared out
// over the CTAs, and how a row's result is written.
#pragma once

#include "kv.cuh"

namespace fp8la {
namespace kv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The two kernels' tiles, and what an item costs beside them, in tiles (measured beside
// the kernels).  Each counts the other's work, too: a call that has too much of either
// writes nothing.
constexpr int kTileTokens = 128;
constexpr int kFewItemRows = 16, kFewItemCost = 4;
constexpr int kManyItemRows = 256, kManyItemCost = 3;

// A partial result that a later kernel joins with the others of its item.
struct Desc {
  int32_t s, h, rt;   // sequence, K/V head, row tile
  int32_t parts;      // CTAs that share it, this one the first; 0: none
};

struct AttnArgs {
  Rows rows;
  Cache cache;
  const void *q;             // fp32 or bf16 [T][Hq][D]
  int64_t ldq, ldq_head;
  uint16_t *out;             // bf16 [T][Hq][D]
  int64_t ldo, ldo_head;
  int32_t out_vec;           // out can be written in 16-byte units
  float *lse;                // [T][ld_lse], natural logarithm; may be null
  int64_t ld_lse;
  int32_t Hq, G, causal;
  int32_t tma;               // whether 16 tokens lie together, as TMA takes them
  // The few-row kernel waits for the kernel before it only where it needs that one's
  // results, and at its end: what it reads was complete when that one began.
  int32_t late;
  Divisor group;             // by G
  float scale_log2;          // of scores, times log2 e
  int64_t row_lo, row_hi;    // rows (tokens times G) of the sequences that are this kernel's
  int64_t max_rows;          // of a segment
  // Shared prefix.  Its own pass takes all rows as one segment (`whole`, S = 1) and
  // writes raw_o, raw_lse; the sequences' pass joins them with its own result.
  const int32_t *whole;      // null, or the word that holds the rows' number
  float *raw_o, *raw_lse;    // [T][Hq][D] and [T][Hq], base 2, or null
  const float *pre_o, *pre_lse;
  const int32_t *prefix_len; // checked by the sequences' pass, too
  int64_t prefix_capacity;
  int32_t prefix_many;       // the prefix's pass was the many-row kernel's
  // Whether the work may pass 2^31 units: of the sequences outside row_lo .. row_hi, which
  // are the other kernel's, and of the prefix.  The host knows what a call's table has room
  // for; counting in every call cost 2 us of instructions fetched.
  int32_t count_other, count_prefix;
  // Partial results: two of each CTA, rows of a tile each.
  float *part_o, *part_lse;
  Desc *desc;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^e with the exponent of v (0 where v is not a positive finite number).
__device__ __forceinline__ int exponent_of(float v) {
  const uint32_t b = __float_as_uint(v);
  const int e = static_cast<int>(b >> 23);  // a sign makes it more than 255
  if (v == 0.0f || e >= 255) return 0;
  return e > 0 ? e - 127 : -126;
}
__device__ __forceinline__ float power_of_two(int e) {  // -126 .. 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// V's scales stand in the exponents, relative to a power of two e0, and a token's share of
// the denominator is its weight over that relative scale.  That holds in FP32 while the
// scales lie within 2^kSpan of e0: what is lost then is 2^-51 of the largest share or less
// (a weight underflows 2^133 below the largest, which is at most 2^kSpan larger by its scale
// than by its share, and the lost one at most 2^kSpan smaller).  A token whose scale is
// smaller keeps its weight, and its share is added up beside, a sum with a maximum of its own
// (set_aside); where a larger one comes, e0 rises to it and what was added up until then
// goes there.  So any positive finite scales are right, and those that an ordinary cache
// holds cost a comparison.
constexpr int kSpan = 40;

// log2 of a scale of any size, relative to 2^e0.
__device__ __forceinline__ float log2_far(float v, int e0) {
  const bool small = v < 1.0f;  // 2^-149 and up: subnormal ones become normal
  return lg2(small ? v * 1.2676506002282294e30f : v) - static_cast<float>((small ? 100 : 0) + e0);
}

// A sum of 2^x as sum * 2^top; adds n * 2^x.  NaN stays.
__device__ __forceinline__ void add_share(float &top, float &sum, float x, float n) {
  const float m = fmaxf(top, x), base = m == -INFINITY ? 0.0f : m;
  // Without shares so far, or of this one, the other's factor is 2^0 or it is not finite.
  const float down = top == -INFINITY ? 0.0f : ex2(top - base);
  sum = sum * down + (x == -INFINITY ? n * 0.0f : n * ex2(x - base));
  top = m;
}

// A row's logarithm, and the two factors (to be applied one after the other, as their
// product may leave FP32's range) that make its result of sums of weights times codes:
// `sum` shares relative to 2^top, `far_sum` relative to 2^far_top, scales relative to 2^e0.
struct Total {
  float lse, f0, f1;
};
static __device__ __noinline__ Total total_with_far(float top, float sum, float far_top, float far_sum,
                                                    int e0) {
  add_share(far_top, far_sum, top, sum);
  const float lse = far_top + lg2(far_sum);
  // top is -inf where no weight was more than 0.
  const float f = ex2(0.5f * (top - lse + static_cast<float>(e0)));
  return {lse, f, f};
}
__device__ __forceinline__ Total total_of(float top, float sum, float far_top, float far_sum,
                                          int e0) {
  if (far_sum == 0.0f) {
    const bool some = sum > 0.0f || sum != sum;
    return {some ? top + lg2(sum) : -INFINITY, some ? rcp(sum) : 0.0f, power_of_two(e0)};
  }
  return total_with_far(top, sum, far_top, far_sum, e0);
}

// A part's weight is 2^x, x <= 0.  Below 2^-126, where FP32 ends, the part still counts if
// its values, by V's scales, are as much larger than the others': then a half of the
// exponent is in the weight and the other half is applied to the values first.
__device__ __forceinline__ bool far_below(float x) { return x < -100.0f && x > -INFINITY; }

// m16n8k16 with half operands.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// One sequence of the call: rows row0 .. row0+n-1, len tokens.
struct Seq {
  int row0, n, len;
};
__device__ __forceinline__ Seq load_seq(const AttnArgs &a, int s) {
  if (a.whole) return {0, *a.whole, *a.rows.lens};
  const int lo = a.rows.offsets[s];
  return {lo, a.rows.offsets[s + 1] - lo, a.rows.lens[s]};
}

// Tokens that rows up to `row` (token times G + head) of a sequence see.
__device__ __forceinline__ int tokens_seen(const AttnArgs &a, const Seq &q, int row) {
  if (!a.causal) return q.len;
  const int end = q.len - q.n + divide(row, a.group) + 1;
  return end < 0 ? 0 : end > q.len ? q.len : end;
}

// Tiles of BN tokens that row tile rt of BM rows goes through, one at least.
template <int BM, int BN>
__device__ __forceinline__ int tiles_of(const AttnArgs &a, const Seq &q, int rt) {
  const int last = min((rt + 1) * BM, q.n * a.G) - 1;
  const int seen = tokens_seen(a, q, last);
  return seen > 0 ? (seen - 1) / BN + 1 : 1;
}

// y / m for y >= 0, 0 < m < 2^31; nearly always of 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t y, uint32_t m) {
  if (static_cast<uint64_t>(y) >> 32 == 0) return static_cast<uint32_t>(y) / m;
  return y / m;
}

// Sum over i < n of floor((x i + b) / m), x, b >= 0, m > 0: whole parts first, then
// the lattice points under the line counted along the other axis.
__device__ __forceinline__ int64_t floor_sum(int64_t n, uint32_t m, uint32_t x, int64_t b) {
  int64_t sum = 0;
#pragma unroll 1
  for (;;) {
    const int64_t whole = quotient(b, m);
    sum += n * (n - 1) / 2 * (x / m) + n * whole;
    x %= m;
    const int64_t y = x * n + (b - whole * m);
    n = quotient(y, m);
    if (n == 0) return sum;
    b = y - n * m;
    const uint32_t t = m;
    m = x;
    x = t;
  }
}

// Units of the row tiles below R of a sequence with `rts` of them: their tiles and COST
// each.  Row tile rt but the
// last one sees len - n + floor(((rt + 1) BM - 1) / G) + 1 tokens, which makes floor((G
// (len - n + BN) + (rt + 1) BM - 1) / (BN G)) tiles, and one where that is less.
template <int BM, int BN, int COST>
__device__ __noinline__ int64_t units_below(const AttnArgs &a, const Seq &q, int rts, int R) {
  if (!a.causal || rts == 1)
    return static_cast<int64_t>(R) * (tiles_of<BM, BN>(a, q, 0) + COST);
  int64_t sum = static_cast<int64_t>(R) * COST;
  if (R == rts) sum += tiles_of<BM, BN>(a, q, --R);
  const int64_t G = a.G, c = static_cast<int64_t>(q.len) - q.n;
  int64_t k = c < 0 ? -G * c / BM : 0;  // BM is a power of two
  if (k > R) k = R;
  return sum + k + floor_sum(R - k, BN * G, BM, G * (c + BN) + (k + 1) * BM - 1);
}

// Row tiles of a sequence; 0 where it has no rows or is another kernel's.
template <int BM>
__device__ __forceinline__ int row_tiles_of(const AttnArgs &a, const Seq &q) {
  const int64_t rows = static_cast<int64_t>(q.n) * a.G;
  if (rows <= 0 || rows < a.row_lo || rows > a.row_hi) return 0;
  return static_cast<int>((rows + BM - 1) / BM);
}

// Units of the sequences that are the other kernel's, whose row tiles have BM rows; each
// thread counts s0 .. s1-1.
template <int THREADS, int BM, int BN, int COST>
__device__ __noinline__ int64_t other_units(const AttnArgs &a, int s0, int s1, int64_t *sums) {
  int64_t sum = 0;
  for (int s = s0; s < s1; ++s) {
    const Seq q = load_seq(a, s);
    const int64_t rows = static_cast<int64_t>(q.n) * a.G;
    if (rows <= 0 || (rows >= a.row_lo && rows <= a.row_hi)) continue;
    const int rts = static_cast<int>((rows + BM - 1) / BM);
    sum += a.cache.heads * units_below<BM, BN, COST>(a, q, rts, rts);
  }
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < THREADS / 32; ++w) sum += sums[w];
  return sum;
}

// Units of the prefix's pass, of `tokens` tokens.
__device__ __forceinline__ int64_t prefix_units(const AttnArgs &a, int tokens) {
  const int64_t rows = static_cast<int64_t>(a.rows.offsets[a.rows.S]) * a.G;
  const int BM = a.prefix_many ? kManyItemRows : kFewItemRows;
  const int cost = a.prefix_many ? kManyItemCost : kFewItemCost;
  const int tiles = tokens > 0 ? (tokens - 1) / kTileTokens + 1 : 1;
  return (rows + BM - 1) / BM * (tiles + cost) * a.cache.heads;
}

struct Share {
  int32_t units, begin, end;   // all units; this CTA's
  int32_t ctas;                // that have work
  int32_t s, h, rt, pos;       // where this CTA begins: unit `pos` of a row tile
};

// Where the range of CTA b begins: floor(units b / ctas).
__device__ __forceinline__ int begin_of(int units, int ctas, int b) {
  const int q = units / ctas;
  return q * b + (units - q * ctas) * b / ctas;
}

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) {
  return __shfl_up_sync(0xffffffffu, v, d);
}

// All units in the order (sequence, K/V head, row tile, then its COST units that are no
// tiles, then its tiles) are cut into equal ranges, one for each CTA: every SM has the
// same work whatever the lengths are.  2^31 units or more (70 TB of codes) are refused, of
// this kernel, of the other one or of the prefix's pass, by all that would write.
// Checks the segments: where they cannot be used, nothing is to be done.
template <int THREADS, int BM, int BN, int COST>
__device__ __noinline__ void share_out(const AttnArgs &a, Share *sh, int64_t *warp_sums) {
  const int S = a.whole ? 1 : a.rows.S;
  const int per = (S + THREADS - 1) / THREADS;
  const int H = a.cache.heads;
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  constexpr bool kMany = BM == kManyItemRows;
  constexpr int kOtherRows = kMany ? kFewItemRows : kManyItemRows;
  constexpr int kOtherCost = kMany ? kFewItemCost : kManyItemCost;
  int64_t sum = 0;
  bool bad = false;
  if (a.prefix_len) {
    const int n = *a.prefix_len;
    bad = n < 0 || n > a.prefix_capacity || (a.count_prefix && prefix_units(a, n) > INT32_MAX);
  }
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const Seq q = load_seq(a, s);
    const bool off = q.row0 < 0 || q.n < 0 || q.n > a.rows.T - q.row0 || q.len < 0 ||
                     q.len > a.rows.capacity || (s == 0 && q.row0 != 0) ||
                     (!a.whole && q.n > a.max_rows);
    bad |= off;
    const int rts = off ? 0 : row_tiles_of<BM>(a, q);
    if (rts > 0) sum += H * units_below<BM, BN, COST>(a, q, rts, rts);
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0) {
      atomicOr(a.rows.status, kStatusBadDeviceArg);
      *sh = {0, 0, 0, 0, 0, 0, 0, 0};
    }
    __syncthreads();
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t run = sum;
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = shfl_up64(run, d);
    if (lane >= d) run += o;
  }
  if (lane == 31) warp_sums[warp] = run;
  __syncthreads();
  int64_t before = run - sum, total = 0;
#pragma unroll 1
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  if (total > INT32_MAX ||
      (a.count_other && other_units<THREADS, kOtherRows, BN, kOtherCost>(a, s0, s1, warp_sums) >
                            INT32_MAX)) {
    if (threadIdx.x == 0) {
      atomicOr(a.rows.status, kStatusBadDeviceArg);
      *sh = {0, 0, 0, 0, 0, 0, 0, 0};
    }
    __syncthreads();
    return;
  }
  const int units = static_cast<int>(total);
  const int ctas = min(units, static_cast<int>(gridDim.x));
  const bool idle = static_cast<int>(blockIdx.x) >= ctas;
  const int begin = idle ? 0 : begin_of(units, ctas, blockIdx.x);
  if (threadIdx.x == 0) {
    sh->units = units;
    sh->begin = begin;
    sh->end = idle ? 0 : begin_of(units, ctas, blockIdx.x + 1);
    sh->ctas = ctas;
  }
  if (!idle && begin >= before && begin < before + sum) {
    // The row tile that holds the unit: the last one with no more units below it.
#pragma unroll 1
    for (int s = s0;; ++s) {
      const Seq q = load_seq(a, s);
      const int rts = row_tiles_of<BM>(a, q);
      if (rts == 0) continue;
      const int each = static_cast<int>(units_below<BM, BN, COST>(a, q, rts, rts));
      if (begin >= before + static_cast<int64_t>(H) * each) {
        before += static_cast<int64_t>(H) * each;
        continue;
      }
      const int at = begin - static_cast<int>(before), h = at / each, left = at - h * each;
      int lo = 0, hi = rts - 1;
#pragma unroll 1
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (units_below<BM, BN, COST>(a, q, rts, mid) <= left) lo = mid;
        else hi = mid - 1;
      }
      sh->s = s;
      sh->h = h;
      sh->rt = lo;
      sh->pos = lo == 0 ? left : left - static_cast<int>(units_below<BM, BN, COST>(a, q, rts, lo));
      break;
    }
  }
  __syncthreads();
}

// The CTA whose range holds unit u.
__device__ __forceinline__ int owner_of(const Share &sh, int u) {
  int b = static_cast<int>(static_cast<float>(u) * sh.ctas / sh.units);
  b = min(max(b, 0), sh.ctas - 1);
  while (begin_of(sh.units, sh.ctas, b) > u) --b;
  while (b + 1 < sh.ctas && begin_of(sh.units, sh.ctas, b + 1) <= u) ++b;
  return b;
}

// Tiles tile0 .. tile0+count-1 of the `tiles` of a row tile with `rows` rows, whose last
// unit, among all units, is the one before `end`.
//
// The tensor cores cut the sums that they hold, by up to 2^-23 for every 16 tokens, and all
// the same way.  So a CTA's part of a row tile, which begins with tile `first`, goes
// through in pieces, an item each, of kPiece tiles at most (four times as many where four
// warps share the tokens): what those before it made (`after` them) lies in the workspace,
// where the part's result will, and is joined with the piece's own.  In one piece, values of
// one sign came out 7.7e-4 too small over 131072 tokens and, with few rows, 1.7e-3 over 2^20;
// a piece of 32768 tokens (of a warp's) loses 2^-12 at most.  A piece costs what an item
// costs: 512 rows after 131072 tokens take 2367 us in one, 2457 in pieces of 256 tiles, 2550
// of 128.
struct Item {
  Seq q;
  int s, h, rt, tile0, count, tiles, rows, end, first;
  bool after, more;   // pieces of the part before this one, and behind it
};
constexpr int kPiece = 256;

// Walks through a CTA's items.
struct Walk {
  int at, end, s, h, rt, pos, rts, first;
  bool after;
  Seq q;
};
template <int BM>
__device__ __noinline__ void start_walk(const AttnArgs &a, const Share &sh, Walk *w) {
  w->at = sh.begin;
  w->end = sh.end;
  w->s = sh.s;
  w->h = sh.h;
  w->rt = sh.rt;
  w->pos = sh.pos;
  w->after = false;
  if (w->at < w->end) {
    w->q = load_seq(a, w->s);
    w->rts = row_tiles_of<BM>(a, w->q);
  }
}
template <int BM, int BN, int COST, int PIECE>
__device__ __noinline__ bool next_item(const AttnArgs &a, Walk *w, Item *it) {
  // A range that ends before a row tile's first tile leaves it to the next CTA.
  const int left = w->end - w->at;
  if (left <= 0 || w->pos + left <= COST) return false;
  if (w->rt >= w->rts) {
    w->rt = 0;
    if (++w->h >= a.cache.heads) {
      w->h = 0;
      do {
        w->q = load_seq(a, ++w->s);
        w->rts = row_tiles_of<BM>(a, w->q);
      } while (w->rts == 0);
    }
  }
  const int tiles = tiles_of<BM, BN>(a, w->q, w->rt);
  const int tile0 = w->pos > COST ? w->pos - COST : 0;
  const int rest = COST + tiles - w->pos;
  int mine = min(rest, left);
  it->q = w->q;
  it->s = w->s;
  it->h = w->h;
  it->rt = w->rt;
  it->tile0 = tile0;
  it->tiles = tiles;
  it->end = w->at + rest;
  it->count = w->pos + mine - COST - tile0;
  it->rows = min(BM, w->q.n * a.G - w->rt * BM);
  it->after = w->after;
  it->first = w->after ? w->first : tile0;
  it->more = it->count > PIECE;
  if (it->more) {
    mine -= it->count - PIECE;
    it->count = PIECE;
  }
  w->at += mine;
  w->after = it->more;
  w->first = it->first;
  w->pos = it->more ? w->pos + mine : 0;
  w->rt += it->more ? 0 : 1;
  return true;
}

// Where and how much a joined row weighs: own result and the prefix's.
struct Weights {
  float own, pre, lse;  // lse: base 2, of both
  float far;            // less than 1: applied first to the side that far_below is about
};
__device__ __forceinline__ Weights weigh(float lse, float p) {
  // A maximum drops a NaN, which the weights and the logarithm are to keep.
  if (lse == -INFINITY && p == -INFINITY) return {0.0f, 0.0f, -INFINITY, 1.0f};
  const float top = fmaxf(lse, p);
  float x = ex2(lse - top), y = ex2(p - top), far = 1.0f;
  const float inv = rcp(x + y), all = top + lg2(x + y);
  if (far_below(lse - top)) x = far = ex2(0.5f * (lse - top));
  if (far_below(p - top)) y = far = ex2(0.5f * (p - top));
  return {x * inv, y * inv, all, far};
}
__device__ __forceinline__ Weights weigh(const AttnArgs &a, int64_t t, int hq, float lse) {
  if (!a.pre_lse) return {1.0f, 0.0f, lse, 1.0f};
  return weigh(lse, a.pre_lse[t * a.Hq + hq]);
}
__device__ __forceinline__ float joined(const Weights &w, float own, float pre) {
  if (w.far < 1.0f) (w.own < w.pre ? own : pre) *= w.far;
  return own * w.own + pre * w.pre;
}

// Writes N consecutive elements of a row's result, own ones in o, and where `d` is 0
// its logarithm.
template <int N>
__device__ __forceinline__ void emit(const AttnArgs &a, int64_t t, int hq, int d,
                                     const float (&o)[N], float lse, const Weights &w) {
  if (a.raw_o) {
    float *p = a.raw_o + (t * a.Hq + hq) * a.cache.D + d;
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = o[i];
    if (d == 0) a.raw_lse[t * a.Hq + hq] = lse;
    return;
  }
  uint16_t *p = a.out + t * a.ldo + hq * a.ldo_head + d;
  const float *q = a.pre_o ? a.pre_o + (t * a.Hq + hq) * a.cache.D + d : nullptr;
  uint32_t u[N / 2];
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    // A side without tokens has weight 0 and zeros.
    const float x = q ? joined(w, o[i], q[i]) : o[i];
    const float y = q ? joined(w, o[i + 1], q[i + 1]) : o[i + 1];
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    u[i / 2] = *reinterpret_cast<const uint32_t *>(&b);
  }
  if (a.out_vec && N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; i += 4)
      *reinterpret_cast<uint4 *>(p + 2 * i) = make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = static_cast<uint16_t>(u[i / 2] >> (16 * (i & 1)));
  }
  if (d == 0 && a.lse) a.lse[t * a.ld_lse + hq] = w.lse * kLn2;
}

fp8la_status launch_many(const AttnArgs &a, bool f32, int format, int ctas, cudaStream_t s);

}  // namespace kv
}  // namespace fp8la

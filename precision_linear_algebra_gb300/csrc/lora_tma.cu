// The adapters' long sums on the 5th-generation tensor cores, BF16 operands and,
// in shrink, FP32 ones too:
// V of rows (shrink) and the factors' gradients (outer); see lora.cu for the
// formulas.
//
// Bound: X (x or dy) once from HBM.  mma.sync reaches 600 TFLOP/s here and its
// fragments cost issue slots, which at ranks above 16 is more than the memory
// time; tcgen05.mma takes both operands from shared memory as TMA left them.
//
// shrink: D[128 rows][R] += X[128][64 k] P[R][64 k]^T, both K-major.  K is
// shared out over a cluster, whose CTAs' sums are added through distributed
// shared memory in rank order.  A CTA's sum is made of short ones of 16 steps
// (kChain), in two accumulators in turn.
//
// expand: D[128 rows][256 columns] = V[128][R] P[R][256 columns], V split into
// two BF16 terms by converter warps (K-major), P as TMA writes it (MN-major).
// base comes by TMA, the epilogue adds to it in shared memory and TMA stores
// the sum from there, so nothing but the sum itself takes an instruction for
// each element: the mma.sync form needs 22 of them and is bound by that.  The
// CTAs get equal shares of the rows of all column blocks.
//
// outer: D[128 columns][R] += X[t][128 columns]^T V[t][R], t being the MMA's
// K.  X is the transposed (MN-major) operand, just as TMA writes a box of 64
// columns x 64 rows.  V (FP32) enters as three BF16 terms, which converter
// warps write K-major ([R][64 t]).  The first term's sums are short ones, as in
// shrink; the other two, 2^-8 of it or less, have an accumulator to themselves.
// Rows past a segment's end belong to other requests and may hold anything, so
// the converters overwrite those that a 16-row MMA step would touch with zeros.
//
// Measured, caches cold, each kernel by itself: shrink of 4096 x 8192, rank 64,
// 23.2 us (70 MB read, 3.0 TB/s, tensor pipe 7.5 %: 148 CTAs, one wave, whose start
// and join are half of it); expand to 4096 x 10240, rank 64, 37.6 us (168 MB in
// and out, 4.5 TB/s); outer of 4096 x 8192 twice, rank 32, three adapters, 51.9 us
// (135 MB, 2.6 TB/s, tensor pipe 10 %).  Of outer with one long chain, 47.9 us:
// its stages of 32 KB took 1.4 us each, 1.1 of it from operands to the commit,
// because X as the transposed M side of the MMA runs at half rate.  X as the N
// side and equal shares of all stages for the SMs streamed at HBM's rate, but
// start, drain and join for 5 us each: 105 us against 97 for that backward pass,
// 139 against 145 at rank 64, 6 to 27 us more for smaller ones, so the simpler
// form stays.
#include "lora.cuh"

namespace fp8la {
namespace lora {
namespace {

// D[tmem] (+)= A[smem] * B[smem]^T, BF16 x BF16 -> F32, one elected thread.
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t adesc,
                                          uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor for kind::f16: BF16 A and B, F32 accumulator.
//   bits 4-5 D format (1 = F32)    bits 7-9, 10-12 A, B format (1 = BF16)
//   bit 15 A is MN-major           bits 17-22 N >> 3, 24-28 M >> 4
__host__ __device__ constexpr uint32_t idesc_bf16_f32(uint32_t M, uint32_t N,
                                                      bool a_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) |
         ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Descriptor of an MN-major operand of 64-element (128-byte) swizzled rows, a
// row for each K: 8-row groups 1024 bytes apart, 64-element blocks
// `block_bytes` apart.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr,
                                                       uint32_t block_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(block_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// 16 TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&u)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3]), "=f"(u[4]), "=f"(u[5]),
        "=f"(u[6]), "=f"(u[7]), "=f"(u[8]), "=f"(u[9]), "=f"(u[10]),
        "=f"(u[11]), "=f"(u[12]), "=f"(u[13]), "=f"(u[14]), "=f"(u[15])
      : "r"(addr)
      : "memory");
}

// ------------------------------------------------------------------- shrink
constexpr int kSThreads = 192;      // warps 0-3 epilogue, 4 producer, 5 MMA
constexpr int kSRows = 128;
constexpr int kSK = 128;            // K of a stage: two boxes of 64
// Stages of one accumulator.  The tensor core cuts off a little of the running
// sum with each addition, always towards zero, so long sums are kept in short
// ones, which the epilogue adds with rounding while the next is made: after 128
// steps of 16 products V's relative error was 2e-6, more than FP32 has.
constexpr int kChain = 2;

// Tile row sums of a shrink CTA, `red` in every CTA of the cluster, to V.
template <int THREADS>
__device__ __forceinline__ void store_v(const ShrinkArgs &a, const Found &f,
                                        const float *red, uint32_t red_addr, int ld) {
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();
  const float alpha = a.alpha ? a.alpha[f.id] : 1.0f;
  const int cells = f.rows * a.R;
  if (csize > 1) cluster_sync_all();
  for (int i = static_cast<int>(crank) * THREADS + threadIdx.x; i < cells;
       i += static_cast<int>(csize) * THREADS) {
    const int r = i / a.R, j = i - r * a.R;
    const float v = csize > 1 ? cluster_sum(red_addr + 4u * (r * ld + j), csize)
                              : red[r * ld + j];
    a.V[(f.row0 + static_cast<int64_t>(r)) * a.ldv + j] = v * alpha;
  }
  if (csize > 1) cluster_sync_all();  // no CTA leaves while its sums are read
}

// RP ranks, a multiple of 16.
template <int RP>
struct ShrinkTma {
  static constexpr int kX = kSRows * kSK * 2;
  static constexpr int kP = RP * kSK * 2;
  static constexpr int kStage = kX + kP;
  static constexpr int STAGES = 4 * kStage <= 200 * 1024 ? 4 : 3;
  static constexpr int kTmemCols = 2 * RP;  // two accumulators
  static constexpr int kLdR = RP + 1;  // of the sums, in floats
  static constexpr int kBar = STAGES * kStage;
  static constexpr int kMisc = kBar + (2 * STAGES + 5) * 8;
  static constexpr int kAlloc = kMisc + 32 + 1024;
  static_assert(kSRows * kLdR * 4 <= STAGES * kStage, "the sums overlay the ring");
  static_assert(kP % 1024 == 0 && kAlloc <= 226 * 1024, "shared memory");
};

template <int RP>
__global__ void __launch_bounds__(kSThreads)
    lora_shrink_tma_kernel(const __grid_constant__ CUtensorMap tmX,
                           const __grid_constant__ CUtensorMap tmP,
                           const ShrinkArgs a, const uint64_t timeout_ns) {
  using C = ShrinkTma<RP>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int warp_sums[kSThreads / 32];
  __shared__ Found slot;
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *sbase = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const Found f = find_tile<kSThreads>(a.seg, blockIdx.y, kSRows, warp_sums, &slot);
  if (f.rows == 0) return;
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();
  if (f.id < 0) {  // rows without an adapter
    if (crank == 0)
      for (int i = threadIdx.x; i < f.rows * a.R; i += kSThreads)
        a.V[(f.row0 + static_cast<int64_t>(i / a.R)) * a.ldv + i % a.R] = 0.0f;
    return;
  }
  const uint32_t bar0 = base + C::kBar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto accfull_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + b); };
  auto accfree_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 2 + b); };
  const uint32_t done_bar = bar0 + 8u * (2 * C::STAGES + 4);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sbase + C::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + C::kMisc + 4);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accfull_bar(b), 1);
      mbar_init(accfree_bar(b), 4);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int nst = static_cast<int>((a.K + kSK - 1) / kSK);
  const int s0 = static_cast<int>(static_cast<int64_t>(nst) * crank / csize);
  const int s1 = static_cast<int>(static_cast<int64_t>(nst) * (crank + 1) / csize);
  float *red = reinterpret_cast<float *>(sbase);

  if (warp == 4) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0, issued = 0;
      for (int c = s0; c < s1; ++c) {
        if (!mbar_wait(empty_bar(s), ph ^ 1u, timeout_ns, a.seg.status, abort_flag))
          break;
        const uint32_t d = base + s * C::kStage;
        mbar_arrive_expect_tx(full_bar(s), C::kStage);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tma_load_2d(d + h * (C::kX / 2), &tmX, full_bar(s), c * kSK + 64 * h, f.row0);
          tma_load_3d(d + C::kX + h * (C::kP / 2), &tmP, full_bar(s),
                      c * kSK + 64 * h, 0, f.id);
        }
        ++issued;
        if (++s == C::STAGES) { s = 0; ph ^= 1u; }
      }
      for (uint32_t st = 0; st < C::STAGES; ++st) {
        if (issued <= st) break;
        const uint32_t arms = (issued - 1 - st) / C::STAGES + 1;
        mbar_wait_drain(full_bar(st), (arms - 1) & 1u, timeout_ns, a.seg.status);
      }
    }
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kSRows, RP, false);
      uint32_t s = 0, ph = 0;
      for (int c = s0; c < s1; ++c) {
        const int g = (c - s0) / kChain, b = g & 1;
        const bool first = (c - s0) % kChain == 0;
        if ((first && !mbar_wait(accfree_bar(b), ((g >> 1) & 1u) ^ 1u, timeout_ns,
                                 a.seg.status, abort_flag)) ||
            !mbar_wait(full_bar(s), ph, timeout_ns, a.seg.status, abort_flag))
          break;
        tc_fence_after();
        const uint32_t d = base + s * C::kStage;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t ad = smem_desc_k128_sw128(d + h * (C::kX / 2));
          const uint64_t bd = smem_desc_k128_sw128(d + C::kX + h * (C::kP / 2));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(tmem_base + b * RP, ad + 2u * k, bd + 2u * k, idesc,
                      (!first || h > 0 || k > 0) ? 1u : 0u);
        }
        umma_commit(empty_bar(s));
        if ((c - s0) % kChain == kChain - 1 || c + 1 == s1) umma_commit(accfull_bar(b));
        if (++s == C::STAGES) { s = 0; ph ^= 1u; }
      }
      umma_commit(done_bar);
      mbar_wait_drain(done_bar, 0, timeout_ns, a.seg.status);
    }
  } else {
    const int row = 32 * warp + lane;
    const uint32_t col0 = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
    float sum[RP];
#pragma unroll
    for (int j = 0; j < RP; ++j) sum[j] = 0.0f;
    const int chains = (s1 - s0 + kChain - 1) / kChain;
    bool ok = true;
    for (int g = 0; g < chains; ++g) {
      const int b = g & 1;
      const bool ready = mbar_wait(accfull_bar(b), (g >> 1) & 1u, timeout_ns,
                                   a.seg.status, abort_flag);
      if (!__all_sync(0xffffffffu, ready)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < RP; j += 16) {
        float v[16];
        tmem_ld16(col0 + b * RP + j, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[j + i] += v[i];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(accfree_bar(b));
    }
    // The ring is free, as the last MMA is done: the sums go there.
    if (ok) {
#pragma unroll
      for (int j = 0; j < RP; ++j) red[row * C::kLdR + j] = sum[j];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
  __syncwarp();
  store_v<kSThreads>(a, f, red, base, C::kLdR);
}

// ------------------------------------------------------------- FP32 shrink
// X in FP32: converter warps split each stage into three BF16 terms, as TMA
// would have written them (K-major, swizzled), and the MMA adds all three.
//
// Bound: X once from HBM; 300 instructions of a converter thread for a stage of
// 32 KB and twelve MMAs stay below the stage's share of memory time.  With a
// forward pass of 4096 rows, rank 64, 8192 -> 8192 it takes 73 us on the stream
// (276 MB, 3.8 TB/s), with the mma.sync form 131.
constexpr int kFConv = 8;           // converter and epilogue warps
constexpr int kFThreads = 32 * (kFConv + 2);
constexpr int kFK = 64;             // K of a stage: two boxes of 32 floats
constexpr int kFChain = 4;          // stages of an accumulator, see kChain

template <int RP>
struct ShrinkF32 {
  static constexpr int kBox = kSRows * 128;
  static constexpr int kX = 2 * kBox;
  static constexpr int kP = RP * 128;
  static constexpr int kStage = kX + kP;
  static constexpr int kTerm = kSRows * 128;
  static constexpr int STAGES = RP <= 64 ? 3 : 2;
  // Two accumulators for the first term, and one for all of the other two, which
  // are 2^-8 of it or less.
  static constexpr int kTmemCols = 4 * RP;          // a power of two
  // Warps that add them up, and the columns of each: half, but no less than a load.
  static constexpr int kAddWarps = RP >= 32 ? kFConv : kFConv / 2;
  static constexpr int kAddCols = RP >= 32 ? RP / 2 : RP;
  static constexpr int kLdR = RP + 1;
  static constexpr int kT = STAGES * kStage;        // [2][3 terms]
  static constexpr int kBar = kT + 6 * kTerm;
  static constexpr int kMisc = kBar + (2 * STAGES + 9) * 8;
  static constexpr int kAlloc = kMisc + 32 + 1024;
  static_assert(kSRows * kLdR * 4 <= kT, "the sums overlay the ring");
  static_assert(kP % 1024 == 0 && kAlloc <= 226 * 1024, "shared memory");
  static_assert(kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM");
};

template <int RP>
__global__ void __launch_bounds__(kFThreads, 1)
    lora_shrink_f32_kernel(const __grid_constant__ CUtensorMap tmX,
                           const __grid_constant__ CUtensorMap tmP,
                           const ShrinkArgs a, const uint64_t timeout_ns) {
  using C = ShrinkF32<RP>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int warp_sums[kFThreads / 32];
  __shared__ Found slot;
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *sbase = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const Found f = find_tile<kFThreads>(a.seg, blockIdx.y, kSRows, warp_sums, &slot);
  if (f.rows == 0) return;
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();
  if (f.id < 0) {  // rows without an adapter
    if (crank == 0)
      for (int i = threadIdx.x; i < f.rows * a.R; i += kFThreads)
        a.V[(f.row0 + static_cast<int64_t>(i / a.R)) * a.ldv + i % a.R] = 0.0f;
    return;
  }
  const uint32_t bar0 = base + C::kBar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto tready_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + b); };
  auto tfree_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 2 + b); };
  auto accfull_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 4 + b); };
  auto accfree_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 6 + b); };
  const uint32_t done_bar = bar0 + 8u * (2 * C::STAGES + 8);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sbase + C::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + C::kMisc + 4);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tready_bar(b), kFConv);
      mbar_init(tfree_bar(b), 1);
      mbar_init(accfull_bar(b), 1);
      mbar_init(accfree_bar(b), C::kAddWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kFConv + 1) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int nst = static_cast<int>((a.K + kFK - 1) / kFK);
  const int s0 = static_cast<int>(static_cast<int64_t>(nst) * crank / csize);
  const int s1 = static_cast<int>(static_cast<int64_t>(nst) * (crank + 1) / csize);
  float *red = reinterpret_cast<float *>(sbase);

  if (warp == kFConv) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0, issued = 0;
      for (int c = s0; c < s1; ++c) {
        if (!mbar_wait(empty_bar(s), ph ^ 1u, timeout_ns, a.seg.status, abort_flag))
          break;
        const uint32_t d = base + s * C::kStage;
        mbar_arrive_expect_tx(full_bar(s), C::kStage);
        tma_load_2d(d, &tmX, full_bar(s), c * kFK, f.row0);
        tma_load_2d(d + C::kBox, &tmX, full_bar(s), c * kFK + 32, f.row0);
        tma_load_3d(d + C::kX, &tmP, full_bar(s), c * kFK, 0, f.id);
        ++issued;
        if (++s == C::STAGES) { s = 0; ph ^= 1u; }
      }
      for (uint32_t st = 0; st < C::STAGES; ++st) {
        if (issued <= st) break;
        const uint32_t arms = (issued - 1 - st) / C::STAGES + 1;
        mbar_wait_drain(full_bar(st), (arms - 1) & 1u, timeout_ns, a.seg.status);
      }
    }
  } else if (warp == kFConv + 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kSRows, RP, false);
      uint32_t s = 0, ph = 0;
      for (int c = s0; c < s1; ++c) {
        const uint32_t b = (c - s0) & 1u, use = (c - s0) >> 1;
        const int g = (c - s0) / kFChain;
        const bool first = (c - s0) % kFChain == 0;
        if ((first && !mbar_wait(accfree_bar(g & 1), ((g >> 1) & 1u) ^ 1u, timeout_ns,
                                 a.seg.status, abort_flag)) ||
            !mbar_wait(full_bar(s), ph, timeout_ns, a.seg.status, abort_flag) ||
            !mbar_wait(tready_bar(b), use & 1u, timeout_ns, a.seg.status, abort_flag))
          break;
        tc_fence_after();
        const uint64_t bd = smem_desc_k128_sw128(base + s * C::kStage + C::kX);
        const uint32_t terms = base + C::kT + 3 * b * C::kTerm;
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          const uint64_t ad = smem_desc_k128_sw128(terms + t * C::kTerm);
          const uint32_t d = tmem_base + (t == 0 ? g & 1 : 2) * RP;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(d, ad + 2u * k, bd + 2u * k, idesc,
                      (k > 0 || t > 1 || (t == 0 ? !first : c > s0)) ? 1u : 0u);
        }
        umma_commit(empty_bar(s));
        umma_commit(tfree_bar(b));
        if ((c - s0) % kFChain == kFChain - 1 || c + 1 == s1)
          umma_commit(accfull_bar(g & 1));
        if (++s == C::STAGES) { s = 0; ph ^= 1u; }
      }
      umma_commit(done_bar);
      mbar_wait_drain(done_bar, 0, timeout_ns, a.seg.status);
    }
  } else {
    // A unit is 8 values of a row: 32 bytes in, 16 bytes of each term out.  A
    // warp takes the same unit of 32 rows, which the swizzle spreads over the
    // banks.
    // They also add the accumulators up, thread = row: a chain's while the second
    // stage after it is multiplied, so that they rarely wait for it.
    float sum[C::kAddCols];
#pragma unroll
    for (int j = 0; j < C::kAddCols; ++j) sum[j] = 0.0f;
    const int first_col = (warp >> 2) * C::kAddCols;
    const uint32_t col0 =
        tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + first_col;
    auto add = [&](int acc) {
#pragma unroll
      for (int j = 0; j < C::kAddCols; j += 16) {
        float v[16];
        tmem_ld16(col0 + acc * RP + j, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[j + i] += v[i];
      }
    };
    auto add_chain = [&](int g) {
      const bool ready = mbar_wait(accfull_bar(g & 1), (g >> 1) & 1u, timeout_ns,
                                   a.seg.status, abort_flag);
      if (!__all_sync(0xffffffffu, ready)) return false;
      tc_fence_after();
      add(g & 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(accfree_bar(g & 1));
      return true;
    };
    int added = 0;
    uint32_t s = 0, ph = 0;
    bool ok = true;
    for (int c = s0; c < s1; ++c) {
      const uint32_t b = (c - s0) & 1u, use = (c - s0) >> 1;
      const bool ready =
          mbar_wait(tfree_bar(b), (use & 1u) ^ 1u, timeout_ns, a.seg.status,
                    abort_flag) &&
          mbar_wait(full_bar(s), ph, timeout_ns, a.seg.status, abort_flag);
      if (!__all_sync(0xffffffffu, ready)) {
        ok = false;
        break;
      }
      const uint32_t row = threadIdx.x % kSRows, first = threadIdx.x / kSRows;
      const uint8_t *x = sbase + s * C::kStage + row * 128;
      const uint32_t out = base + C::kT + 3 * b * C::kTerm + row * 128;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t unit = first + 2 * u;   // of 8 in a row
        const uint8_t *p = x + (unit >> 2) * C::kBox;
        const uint32_t q = 2 * (unit & 3u);
        const float4 lo = *reinterpret_cast<const float4 *>(p + ((q ^ (row & 7u)) << 4));
        const float4 hi =
            *reinterpret_cast<const float4 *>(p + (((q + 1) ^ (row & 7u)) << 4));
        uint32_t w[4][3];
        split_pair<3>(lo.x, lo.y, w[0]);
        split_pair<3>(lo.z, lo.w, w[1]);
        split_pair<3>(hi.x, hi.y, w[2]);
        split_pair<3>(hi.z, hi.w, w[3]);
#pragma unroll
        for (int t = 0; t < 3; ++t)
          st_shared_v4(out + t * C::kTerm + ((unit ^ (row & 7u)) << 4), w[0][t], w[1][t],
                       w[2][t], w[3][t]);
      }
      if (++s == C::STAGES) { s = 0; ph ^= 1u; }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(tready_bar(b));
      if (warp < C::kAddWarps && c - s0 == (added + 1) * kFChain + 1) {
        if (!add_chain(added)) {
          ok = false;
          break;
        }
        ++added;
      }
    }
    if (warp < C::kAddWarps) {
      const int chains = (s1 - s0 + kFChain - 1) / kFChain;
      for (; ok && added < chains; ++added) ok = add_chain(added);
      // The ring is free, as the last MMA is done: the sums go there.
      if (ok) {
        if (chains > 0) add(2);
        const int row = 32 * (warp & 3) + lane;
#pragma unroll
        for (int j = 0; j < C::kAddCols; ++j)
          red[row * C::kLdR + first_col + j] = sum[j];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kFConv + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
  __syncwarp();
  store_v<kFThreads>(a, f, red, base, C::kLdR);
}

// ------------------------------------------------------------------- expand
constexpr int kEEpi = 8;            // epilogue warps
constexpr int kEConv = 4;           // warps that split V
constexpr int kEProducer = kEEpi + kEConv;
constexpr int kEMma = kEProducer + 1;
constexpr int kEStore = kEProducer + 2;
constexpr int kEThreads = 32 * (kEStore + 1);
constexpr int kECols = 256;
constexpr int kERows = 128;         // of a tile
constexpr int kEGrain = 64;         // rows by which the CTAs' shares are cut

template <int RP>
struct ExpandTma {
  static constexpr int kBox = kERows * 128;         // 128 rows x 64 columns
  static constexpr int kStage = 4 * kBox;
  static constexpr int kPBox = RP * 128;            // RP ranks x 64 columns
  static constexpr int kVTerm = kERows * 128;       // 128 rows x up to 64 ranks
  static constexpr int kP = 2 * kStage;
  static constexpr int kV = kP + 4 * kPBox;
  static constexpr int kBar = kV + 2 * kVTerm;
  static constexpr int kNumBars = 15;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kSegs = kMisc + 16;
  static constexpr int kAlloc = kSegs + (2 * kMaxSegments + 1) * 4 + 1024;
  static constexpr int kUnits = kERows * (RP / 8) / (32 * kEConv);
  static_assert(kPBox % 1024 == 0 && kBar % 8 == 0, "swizzle atoms");
  static_assert(kAlloc <= 226 * 1024, "shared memory");
};

template <int RP>
__global__ void __launch_bounds__(kEThreads, 1)
    lora_expand_tma_kernel(const __grid_constant__ CUtensorMap tmBase,
                           const __grid_constant__ CUtensorMap tmOut,
                           const __grid_constant__ CUtensorMap tmP,
                           const ExpandArgs a, const uint64_t timeout_ns) {
  using C = ExpandTma<RP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *sbase = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int *offsets = reinterpret_cast<int *>(sbase + C::kSegs);
  int *ids = offsets + a.seg.S + 1;
  const uint32_t bar0 = base + C::kBar;
  auto full_bar = [&](int b) { return bar0 + 8u * b; };          // base is there
  auto empty_bar = [&](int b) { return bar0 + 8u * (2 + b); };   // and stored
  auto done_bar = [&](int b) { return bar0 + 8u * (4 + b); };    // out is staged
  auto accfull_bar = [&](int b) { return bar0 + 8u * (6 + b); };
  auto accfree_bar = [&](int b) { return bar0 + 8u * (8 + b); };
  const uint32_t pfull_bar = bar0 + 80, pfree_bar = bar0 + 88;
  const uint32_t vready_bar = bar0 + 96, vfree_bar = bar0 + 104;
  const uint32_t final_bar = bar0 + 112;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sbase + C::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + C::kMisc + 4);
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(full_bar(b), 1);
      mbar_init(empty_bar(b), 1);
      mbar_init(done_bar(b), kEEpi);
      mbar_init(accfull_bar(b), 1);
      mbar_init(accfree_bar(b), kEEpi);
    }
    mbar_init(pfull_bar, 1);
    mbar_init(pfree_bar, 1);
    mbar_init(vready_bar, kEConv);
    mbar_init(vfree_bar, 1);
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (!load_segments<kEThreads>(a.seg, offsets, ids)) return;
  if (warp == kEMma) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const bool in_place = a.base == a.out;

  // Every role goes through the same tiles: visit(tile, n) for each, in order;
  // false ends the walk.
  auto tiles = [&](auto &&visit) {
    const int groups = (a.seg.T + kEGrain - 1) / kEGrain;
    const int64_t blocks = (a.N + kECols - 1) / kECols, all = groups * blocks;
    int64_t u = all * blockIdx.x / gridDim.x;
    const int64_t u1 = all * (blockIdx.x + 1) / gridDim.x;
    int n = 0;
    while (u < u1) {
      const int block = static_cast<int>(u / groups);
      const int g0 = static_cast<int>(u - static_cast<int64_t>(block) * groups);
      const int g1 = static_cast<int>(min(static_cast<int64_t>(groups), g0 + u1 - u));
      const int end = min(a.seg.T, g1 * kEGrain);
      Walk w;
      begin_walk(w, g0 * kEGrain, a.seg.S, offsets);
      while (w.row < end) {
        settle_walk<kERows>(w, a.seg.S, offsets, ids, end);
        // Rows without an adapter are where they should be already, in place.
        if (w.id >= 0 || !in_place)
          if (!visit(w, block * kECols, n++)) return;
        w.row += w.n;
      }
      u += g1 - g0;
    }
  };
  // Whether a tile's sums are stored by TMA.  Not those of a tile that ends inside
  // the 128 rows: what follows belongs to another segment or share.  Nor where the
  // matrix ends inside a 16-byte unit: TMA stores whole units, and what follows a
  // row's last column belongs to the caller.
  auto by_tma = [&](const Walk &w, int col) {
    return w.n == kERows && (col + kECols <= a.N || a.N % 8 == 0);
  };
  // Runs of tiles with one factor: its adapter and column block.
  struct Run {
    int id = -1, col = -1, count = 0;
    __device__ bool next(const Walk &w, int c) {
      if (w.id < 0 || (w.id == id && c == col)) return false;
      id = w.id;
      col = c;
      ++count;
      return true;
    }
  };

  if (warp == kEProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      Run run;
      int issued = 0;
      tiles([&](const Walk &w, int col, int n) {
        const int b = n & 1;
        if (run.next(w, col)) {
          if (run.count > 1 && !mbar_wait(pfree_bar, run.count & 1u, timeout_ns,
                                          a.seg.status, abort_flag))
            return false;
          mbar_arrive_expect_tx(pfull_bar, 4 * C::kPBox);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tma_load_3d(base + C::kP + j * C::kPBox, &tmP, pfull_bar, col + 64 * j, 0,
                        w.id);
        }
        if (!mbar_wait(empty_bar(b), ((n >> 1) & 1u) ^ 1u, timeout_ns, a.seg.status,
                       abort_flag))
          return false;
        mbar_arrive_expect_tx(full_bar(b), C::kStage);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tma_load_2d(base + b * C::kStage + j * C::kBox, &tmBase, full_bar(b),
                      col + 64 * j, w.row);
        ++issued;
        return true;
      });
      for (int b = 0; b < 2; ++b)
        if (issued > b)
          mbar_wait_drain(full_bar(b), ((issued - 1 - b) / 2) & 1u, timeout_ns,
                          a.seg.status);
      if (run.count > 0)
        mbar_wait_drain(pfull_bar, (run.count - 1) & 1u, timeout_ns, a.seg.status);
    }
  } else if (warp == kEMma) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kERows, kECols, false) | (1u << 16);
      Run run;
      int m = 0;  // tiles with an adapter
      tiles([&](const Walk &w, int col, int n) {
        if (w.id < 0) return true;
        const int b = m & 1;
        if (run.next(w, col)) {
          // All MMAs with the factor before this one have been issued.
          if (run.count > 1) umma_commit(pfree_bar);
          if (!mbar_wait(pfull_bar, (run.count - 1) & 1u, timeout_ns, a.seg.status,
                         abort_flag))
            return false;
        }
        if (!mbar_wait(accfree_bar(b), ((m >> 1) & 1u) ^ 1u, timeout_ns, a.seg.status,
                       abort_flag) ||
            !mbar_wait(vready_bar, m & 1u, timeout_ns, a.seg.status, abort_flag))
          return false;
        tc_fence_after();
        // V [128 rows][ranks] is K-major; the factor [ranks][columns] MN-major.
#pragma unroll
        for (int k = 0; k < RP / 16; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            umma_bf16(tmem_base + b * kECols,
                      smem_desc_k128_sw128(base + C::kV + t * C::kVTerm) + 2u * k,
                      smem_desc_mn_sw128(base + C::kP + k * 2048, C::kPBox), idesc,
                      (k > 0 || t > 0) ? 1u : 0u);
        umma_commit(vfree_bar);
        umma_commit(accfull_bar(b));
        ++m;
        return true;
      });
      umma_commit(final_bar);
      mbar_wait_drain(final_bar, 0, timeout_ns, a.seg.status);
    }
  } else if (warp == kEStore) {
    // --------------------------------------------------------------- store
    if (lane == 0) {
      tiles([&](const Walk &w, int col, int n) {
        const int b = n & 1;
        if (!mbar_wait(done_bar(b), (n >> 1) & 1u, timeout_ns, a.seg.status, abort_flag))
          return false;
        if (by_tma(w, col)) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col + 64 * j < a.N)
              tma_store_2d(&tmOut, base + b * C::kStage + j * C::kBox, col + 64 * j,
                           w.row);
          bulk_commit_group();
          bulk_wait_read_all();
        }
        mbar_arrive(empty_bar(b));
        return true;
      });
      bulk_wait_all();
    }
  } else if (warp >= kEEpi) {
    // ---------------------------------------------------------- converters
    const int ct = threadIdx.x - 32 * kEEpi;
    float v[C::kUnits][8], alpha = 1.0f;
    // A tile's V is loaded while the one before is multiplied: the buffer is
    // waited for after the loads.
    auto load_v = [&](const Walk &w) {
      alpha = a.alpha ? __ldg(a.alpha + w.id) : 1.0f;
#pragma unroll
      for (int u = 0; u < C::kUnits; ++u) {
        const int e = ct + u * 32 * kEConv;
        const int r = e / (RP / 8), j = 8 * (e % (RP / 8));
        const float *p = a.V + (w.row + static_cast<int64_t>(r)) * a.ldv + j;
        if (a.v_vec && j + 8 <= a.R) {
          float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y = x;
          if (r < w.n) {
            x = __ldcg(reinterpret_cast<const float4 *>(p));
            y = __ldcg(reinterpret_cast<const float4 *>(p) + 1);
          }
          v[u][0] = x.x;
          v[u][1] = x.y;
          v[u][2] = x.z;
          v[u][3] = x.w;
          v[u][4] = y.x;
          v[u][5] = y.y;
          v[u][6] = y.z;
          v[u][7] = y.w;
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            v[u][q] = r < w.n && j + q < a.R ? __ldcg(p + q) : 0.0f;
        }
      }
    };
    auto store_v = [&](int m) {
      const bool ready = mbar_wait(vfree_bar, (m & 1u) ^ 1u, timeout_ns, a.seg.status,
                                   abort_flag);
      if (!__all_sync(0xffffffffu, ready)) return false;
#pragma unroll
      for (int u = 0; u < C::kUnits; ++u) {
        const int e = ct + u * 32 * kEConv;
        const uint32_t r = e / (RP / 8), unit = e % (RP / 8);
        uint32_t t[2][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t x[2];
          split_pair<2>(v[u][2 * q] * alpha, v[u][2 * q + 1] * alpha, x);
          t[0][q] = x[0];
          t[1][q] = x[1];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          st_shared_v4(base + C::kV + k * C::kVTerm + r * 128 +
                           ((unit ^ (r & 7u)) << 4),
                       t[k][0], t[k][1], t[k][2], t[k][3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(vready_bar);
      return true;
    };
    int m = 0;
    tiles([&](const Walk &w, int col, int n) {
      if (w.id < 0) return true;
      load_v(w);
      return store_v(m++);
    });
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = warp >> 2;
    const int row = 32 * quarter + lane;
    const uint32_t lane_base =
        tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 128 * half;
    int m = 0;
    tiles([&](const Walk &w, int col, int n) {
      const int b = n & 1, t = m & 1;
      bool ready = mbar_wait(full_bar(b), (n >> 1) & 1u, timeout_ns, a.seg.status,
                             abort_flag);
      if (w.id >= 0)
        ready = ready && mbar_wait(accfull_bar(t), (m >> 1) & 1u, timeout_ns,
                                   a.seg.status, abort_flag);
      if (!__all_sync(0xffffffffu, ready)) return false;
      tc_fence_after();
      uint16_t *dst = a.out + (w.row + static_cast<int64_t>(row)) * a.ld_out;
      const bool stage = by_tma(w, col);
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {  // 32 columns
        uint8_t *src = sbase + b * C::kStage + (2 * half + (j >> 1)) * C::kBox + row * 128;
        uint32_t acc[32];
        if (w.id >= 0) tmem_ld32(lane_base + t * kECols + 32 * j, acc);
        const int64_t c0 = col + 128 * half + 32 * j;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 8 columns
          uint4 *at = reinterpret_cast<uint4 *>(
              src + (((4 * (j & 1) + i) ^ (row & 7)) << 4));
          uint4 x = *at;
          if (w.id >= 0) {
            uint32_t *y = &x.x;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const __nv_bfloat162 s = __floats2bfloat162_rn(
                  bf_lo(y[q]) + __uint_as_float(acc[8 * i + 2 * q]),
                  bf_hi(y[q]) + __uint_as_float(acc[8 * i + 2 * q + 1]));
              y[q] = *reinterpret_cast<const uint32_t *>(&s);
            }
          }
          if (stage) {
            *at = x;
          } else if (row < w.n) {
            const int64_t c = c0 + 8 * i;
            if (c + 8 <= a.N) {
              *reinterpret_cast<uint4 *>(dst + c) = x;
            } else {
              const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (c + q < a.N)
                  dst[c + q] = static_cast<uint16_t>(q & 1 ? y[q >> 1] >> 16 : y[q >> 1]);
            }
          }
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (w.id >= 0) mbar_arrive(accfree_bar(t));
        mbar_arrive(done_bar(b));
      }
      if (w.id >= 0) ++m;
      return true;
    });
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kEMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// -------------------------------------------------------------------- outer
constexpr int kOConv = 8;           // converter and epilogue warps
constexpr int kOThreads = 32 * (kOConv + 2);
constexpr int kOCols = 256;         // two MMA blocks of 128
constexpr int kORows = 64;          // of a stage
// Stages of an accumulator, see kChain.  4, 8 and 16 take 102.3, 101.8 and 101.5 us
// for the backward pass of outer's figure above; 4 leave 4.3e-7 of dA, 8 6.6e-7.
constexpr int kOChain = 4;

template <int RP>
struct OuterTma {
  static constexpr int kBox = 64 * 128;             // 64 rows x 64 columns
  static constexpr int kX = 4 * kBox;
  static constexpr int kTerm = RP * 128;            // [RP][64 t]
  static constexpr int kV = 3 * kTerm;
  // Two CTAs on an SM for the smallest ranks, so that one streams while the
  // other starts or adds up.
  static constexpr int STAGES = RP <= 32 ? 2 : 3;
  // NACC accumulators for V's first term, and one for all of the other two, which
  // are 2^-8 of it or less.  With one the MMA waits until it has been added up.
  static constexpr int NACC = RP <= 64 ? 2 : 1;
  static constexpr int kTmemCols = RP <= 64 ? 8 * RP : 4 * RP;  // a power of two
  static constexpr int kVBuf = STAGES * kX;         // [2][3 terms]
  static constexpr int kLdR = kOCols + 4;
  static constexpr int kBar = kVBuf + 2 * kV;
  static constexpr int kMisc = kBar + (2 * STAGES + 9) * 8;
  static constexpr int kSegs = kMisc + 32;          // three lists
  static constexpr int kAlloc = kSegs + 3 * kMaxSegments * 4 + 1024;
  static_assert(RP * kLdR * 4 <= kBar, "the sums overlay the ring");
  static_assert(kVBuf % 1024 == 0 && kTerm % 1024 == 0, "swizzle atoms");
  static_assert(kAlloc <= 226 * 1024, "shared memory");
};

// grid: x = cluster rank (rows), y = column block of either side, z = adapter.
template <int RP>
__global__ void __launch_bounds__(kOThreads, RP <= 32 ? 2 : 1)
    lora_outer_tma_kernel(const __grid_constant__ CUtensorMap tm0,
                          const __grid_constant__ CUtensorMap tm1,
                          const OuterArgs a, const uint64_t timeout_ns) {
  using C = OuterTma<RP>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int warp_sums[kOThreads / 32];
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *sbase = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int *seg_lo = reinterpret_cast<int *>(sbase + C::kSegs);
  int *seg_hi = seg_lo + kMaxSegments, *seg_step = seg_hi + kMaxSegments;
  const uint32_t bar0 = base + C::kBar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto vready_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + b); };
  auto vfree_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 2 + b); };
  auto accfull_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 4 + b); };
  auto accfree_bar = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 6 + b); };
  const uint32_t done_bar = bar0 + 8u * (2 * C::STAGES + 8);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sbase + C::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + C::kMisc + 4);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(vready_bar(b), kOConv);
      mbar_init(vfree_bar(b), 1);
      mbar_init(accfull_bar(b), 1);
      mbar_init(accfree_bar(b), kOConv);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  const int adapter = blockIdx.z;
  const uint32_t crank = cluster_ctarank(), csize = cluster_size();

  // The adapter's segments, in order, with the stages before each.
  constexpr int kPer = (kMaxSegments + kOThreads - 1) / kOThreads;
  const int per = (a.seg.S + kOThreads - 1) / kOThreads;
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
        steps += (h - l + kORows - 1) / kORows;
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0) atomicOr(a.seg.status, kStatusBadDeviceArg);
    return;  // every CTA of the grid sees the same
  }
  int nseg, nstep;
  int at = block_exclusive<kOThreads>(mine, warp_sums, &nseg);
  int before = block_exclusive<kOThreads>(steps, warp_sums, &nstep);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (hi[i] > lo[i]) {
      seg_lo[at] = lo[i];
      seg_hi[at] = hi[i];
      seg_step[at] = before;
      ++at;
      before += (hi[i] - lo[i] + kORows - 1) / kORows;
    }
  if (warp == kOConv + 1) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int s0 = static_cast<int>(static_cast<int64_t>(nstep) * crank / csize);
  const int s1 = static_cast<int>(static_cast<int64_t>(nstep) * (crank + 1) / csize);
  const int blocks0 = static_cast<int>((a.side[0].N + kOCols - 1) / kOCols);
  const bool second = static_cast<int>(blockIdx.y) >= blocks0;
  const OuterSide &o = a.side[second];
  const CUtensorMap *tm = second ? &tm1 : &tm0;
  // Without rows the gradient is 0 whatever alpha is.
  const float scale = o.use_alpha && nstep > 0 ? a.alpha[adapter] : 1.0f;
  const int col0 = (blockIdx.y - (second ? blocks0 : 0)) * kOCols;
  // First row and number of rows of stage s; `i` follows s upwards.
  auto rows_of = [&](int s, int &i, int &t0) {
    while (i + 1 < nseg && seg_step[i + 1] <= s) ++i;
    t0 = seg_lo[i] + kORows * (s - seg_step[i]);
    return min(kORows, seg_hi[i] - t0);
  };

  if (warp == kOConv) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t s = 0, ph = 0, issued = 0;
      int i = 0;
      for (int c = s0; c < s1; ++c) {
        if (!mbar_wait(empty_bar(s), ph ^ 1u, timeout_ns, a.seg.status, abort_flag))
          break;
        int t0;
        rows_of(c, i, t0);
        mbar_arrive_expect_tx(full_bar(s), C::kX);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tma_load_2d(base + s * C::kX + j * C::kBox, tm, full_bar(s), col0 + 64 * j, t0);
        ++issued;
        if (++s == C::STAGES) { s = 0; ph ^= 1u; }
      }
      for (uint32_t st = 0; st < C::STAGES; ++st) {
        if (issued <= st) break;
        const uint32_t arms = (issued - 1 - st) / C::STAGES + 1;
        mbar_wait_drain(full_bar(st), (arms - 1) & 1u, timeout_ns, a.seg.status);
      }
    }
  } else if (warp == kOConv + 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, RP, true);
      uint32_t s = 0, ph = 0;
      int i = 0;
      for (int c = s0; c < s1; ++c) {
        const uint32_t b = (c - s0) & 1u, use = (c - s0) >> 1;
        const int g = (c - s0) / kOChain, acc = g % C::NACC;
        const bool first = (c - s0) % kOChain == 0;
        // The converters of a stage have seen its X.
        if ((first && !mbar_wait(accfree_bar(acc), ((g / C::NACC) & 1u) ^ 1u, timeout_ns,
                                 a.seg.status, abort_flag)) ||
            !mbar_wait(full_bar(s), ph, timeout_ns, a.seg.status, abort_flag) ||
            !mbar_wait(vready_bar(b), use & 1u, timeout_ns, a.seg.status, abort_flag))
          break;
        tc_fence_after();
        int t0;
        const int n = rows_of(c, i, t0);
        const uint32_t x = base + s * C::kX;
        const uint32_t v = base + C::kVBuf + b * C::kV;
        for (int k = 0; 16 * k < n; ++k)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint64_t ad =
                smem_desc_mn_sw128(x + 2 * m * C::kBox + k * 2048, C::kBox);
#pragma unroll
            for (int t = 0; t < 3; ++t)
              umma_bf16(tmem_base + ((t == 0 ? acc : C::NACC) * 2 + m) * RP, ad,
                        smem_desc_k128_sw128(v + t * C::kTerm) + 2u * k, idesc,
                        (k > 0 || t > 1 || (t == 0 ? !first : c > s0)) ? 1u : 0u);
          }
        umma_commit(empty_bar(s));
        umma_commit(vfree_bar(b));
        if ((c - s0) % kOChain == kOChain - 1 || c + 1 == s1)
          umma_commit(accfull_bar(acc));
        if (++s == C::STAGES) { s = 0; ph ^= 1u; }
      }
      umma_commit(done_bar);
      mbar_wait_drain(done_bar, 0, timeout_ns, a.seg.status);
    }
  } else {
    // --------------------------------------------- converters and epilogue
    // A unit is one rank's 8 rows: 16 bytes of each term.
    constexpr int kUnits = RP * 8 / (32 * kOConv);
    static_assert(RP * 8 >= 32 * kOConv || RP == 16, "units");
    constexpr int kU = kUnits > 0 ? kUnits : 1;
    uint32_t s = 0, ph = 0;
    int i_load = 0, i_fix = 0;
    float w[kU][8];
    auto load_v = [&](int c) {
      int t0 = 0;
      const int n = c < s1 ? rows_of(c, i_load, t0) : 0;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int e = threadIdx.x + u * 32 * kOConv;
        const int j = e % RP, t = 8 * (e / RP);
        const float *p = o.W + (t0 + static_cast<int64_t>(t)) * o.ldw + j;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          w[u][q] = t + q < n && j < a.R && e < RP * 8 ? __ldcg(p + q * o.ldw) : 0.0f;
      }
    };
    // Thread = column of X; the two halves of the warps have a block each.  A chain
    // is added up while the second stage after it is multiplied, so that they
    // rarely wait for it, or the first, where the MMA waits for them.
    float sum[RP];
#pragma unroll
    for (int j = 0; j < RP; ++j) sum[j] = 0.0f;
    const int m = warp >> 2;
    const uint32_t t_addr =
        tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + m * RP;
    auto add = [&](int acc) {
#pragma unroll
      for (int j = 0; j < RP; j += 16) {
        float v[16];
        tmem_ld16(t_addr + acc * 2 * RP + j, v);
#pragma unroll
        for (int q = 0; q < 16; ++q) sum[j + q] += v[q];
      }
    };
    auto add_chain = [&](int g) {
      const int acc = g % C::NACC;
      const bool ready = mbar_wait(accfull_bar(acc), (g / C::NACC) & 1u, timeout_ns,
                                   a.seg.status, abort_flag);
      if (!__all_sync(0xffffffffu, ready)) return false;
      tc_fence_after();
      add(acc);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(accfree_bar(acc));
      return true;
    };
    int added = 0;
    load_v(s0);
    bool ok = true;
    for (int c = s0; c < s1; ++c) {
      const uint32_t b = (c - s0) & 1u, use = (c - s0) >> 1;
      const bool ready = mbar_wait(vfree_bar(b), (use & 1u) ^ 1u, timeout_ns,
                                   a.seg.status, abort_flag);
      if (!__all_sync(0xffffffffu, ready)) {
        ok = false;
        break;
      }
      const uint32_t v = base + C::kVBuf + b * C::kV;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int e = threadIdx.x + u * 32 * kOConv;
        const uint32_t j = e % RP, unit = e / RP;
        uint32_t t[3][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t p[3];
          split_pair<3>(w[u][2 * q], w[u][2 * q + 1], p);
#pragma unroll
          for (int k = 0; k < 3; ++k) t[k][q] = p[k];
        }
        if (e < RP * 8)
#pragma unroll
          for (int k = 0; k < 3; ++k)
            st_shared_v4(v + k * C::kTerm + j * 128 + ((unit ^ (j & 7u)) << 4), t[k][0],
                         t[k][1], t[k][2], t[k][3]);
      }
      load_v(c + 1);
      int t0;
      const int n = rows_of(c, i_fix, t0);
      if (n % 16 != 0) {
        // Rows n.. of the last MMA step are other requests': zeros instead.
        const bool full = mbar_wait(full_bar(s), ph, timeout_ns, a.seg.status, abort_flag);
        if (!__all_sync(0xffffffffu, full)) {
          ok = false;
          break;
        }
        const int rows = 16 - n % 16;
        for (int e = threadIdx.x; e < rows * 32; e += 32 * kOConv)
          st_shared_v4(base + s * C::kX + (e & 3) * C::kBox + (n + (e >> 5)) * 128 +
                           ((e >> 2) & 7) * 16,
                       0, 0, 0, 0);
      }
      if (++s == C::STAGES) { s = 0; ph ^= 1u; }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(vready_bar(b));
      if (c - s0 == (added + 1) * kOChain + C::NACC - 1) {
        if (!add_chain(added)) {
          ok = false;
          break;
        }
        ++added;
      }
    }
    const int chains = (s1 - s0 + kOChain - 1) / kOChain;
    for (; ok && added < chains; ++added) ok = add_chain(added);
    // The ring is free, as the last MMA is done: the sums go there.
    if (ok) {
      if (chains > 0) add(C::NACC);
      const int cc = 128 * m + 32 * (warp & 3) + lane;
      float *red = reinterpret_cast<float *>(sbase);
#pragma unroll
      for (int j = 0; j < RP; ++j) {
        if (csize > 1)
          red[j * C::kLdR + cc] = sum[j];
        else if (j < a.R && col0 + cc < o.N)
          o.G[(static_cast<int64_t>(adapter) * a.R + j) * o.N + col0 + cc] =
              sum[j] * scale;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kOConv + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
  __syncwarp();
  if (csize == 1) return;
  cluster_sync_all();
  const int cells = a.R * kOCols;
  for (int i = static_cast<int>(crank) * kOThreads + threadIdx.x; i < cells;
       i += static_cast<int>(csize) * kOThreads) {
    const int r = i / kOCols, cc = i % kOCols;
    if (col0 + cc >= o.N) continue;
    o.G[(static_cast<int64_t>(adapter) * a.R + r) * o.N + col0 + cc] =
        cluster_sum(base + 4u * (r * C::kLdR + cc), csize) * scale;
  }
  cluster_sync_all();  // no CTA leaves while its sums are read
}

// --------------------------------------------------------------------- host
// BF16 matrices [outer][rows][width] as swizzled boxes of 64 columns.  The
// stride of a single row, or matrix, is never used and may be anything.
bool encode_bf16(CUtensorMap *m, const void *p, int64_t width, int64_t rows,
                 int64_t outer, int64_t ld, int64_t stride, uint32_t box_rows,
                 int dims_n) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width),
                              static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(outer)};
  if (rows == 1) ld = (width + 7) / 8 * 8;
  if (outer == 1) stride = rows * ld;
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2,
                                 static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims_n, const_cast<void *>(p), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// FP32 matrix [rows][width] as swizzled boxes of 32 columns.
bool encode_f32(CUtensorMap *m, const void *p, int64_t width, int64_t rows, int64_t ld,
                uint32_t box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 4};
  const cuuint32_t box[2] = {32, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(p), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int RP>
fp8la_status shrink_one(const ShrinkArgs &a, int slot, cudaStream_t s) {
  using C = ShrinkTma<RP>;
  auto kern = lora_shrink_tma_kernel<RP>;
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  CUtensorMap tmX, tmP;
  if (!encode_bf16(&tmX, a.X, a.K, a.seg.T, 1, a.ldx, 0, kSRows, 2) ||
      !encode_bf16(&tmP, a.P, a.K, a.R, a.seg.n, a.ldp, a.stride_p, RP, 3))
    return FP8LA_ERR_CUDA;
  const int64_t T = a.seg.T, S = a.seg.S;
  const int64_t tiles = T / kSRows + ((S < T ? S : T) + 1) / 2;
  const int cluster = choose_cluster(tiles, (a.K + kSK - 1) / kSK, sms(), 6);
  return launch(kern, dim3(cluster, static_cast<unsigned>(tile_bound(T, S, kSRows)), 1),
                kSThreads, C::kAlloc, cluster, s, tmX, tmP, a, wait_timeout_ns());
}

template <int RP>
fp8la_status shrink_f32_one(const ShrinkArgs &a, int slot, cudaStream_t s) {
  using C = ShrinkF32<RP>;
  auto kern = lora_shrink_f32_kernel<RP>;
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  CUtensorMap tmX, tmP;
  if (!encode_f32(&tmX, a.X, a.K, a.seg.T, a.ldx, kSRows) ||
      !encode_bf16(&tmP, a.P, a.K, a.R, a.seg.n, a.ldp, a.stride_p, RP, 3))
    return FP8LA_ERR_CUDA;
  const int64_t T = a.seg.T, S = a.seg.S;
  const int64_t tiles = T / kSRows + ((S < T ? S : T) + 1) / 2;
  const int cluster = choose_cluster(tiles, (a.K + kFK - 1) / kFK, sms(), 6);
  return launch(kern, dim3(cluster, static_cast<unsigned>(tile_bound(T, S, kSRows)), 1),
                kFThreads, C::kAlloc, cluster, s, tmX, tmP, a, wait_timeout_ns());
}

template <int RP>
fp8la_status expand_one(const ExpandArgs &a, int slot, cudaStream_t s) {
  using C = ExpandTma<RP>;
  auto kern = lora_expand_tma_kernel<RP>;
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  CUtensorMap tmBase, tmOut, tmP;
  const int sms = sm_count();
  if (sms <= 0 ||
      !encode_bf16(&tmBase, a.base, a.N, a.seg.T, 1, a.ld_base, 0, kERows, 2) ||
      !encode_bf16(&tmOut, a.out, a.N, a.seg.T, 1, a.ld_out, 0, kERows, 2) ||
      !encode_bf16(&tmP, a.P, a.N, a.R, a.seg.n, a.ldp, a.stride_p, RP, 3))
    return FP8LA_ERR_CUDA;
  return launch(kern, dim3(sms, 1, 1), kEThreads, C::kAlloc, 0, s, tmBase, tmOut, tmP, a,
                wait_timeout_ns());
}

template <int RP>
fp8la_status outer_one(const OuterArgs &a, int slot, cudaStream_t s) {
  using C = OuterTma<RP>;
  auto kern = lora_outer_tma_kernel<RP>;
  if (once_per_device(slot, [&] {
        return cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
      }) != cudaSuccess)
    return FP8LA_ERR_CUDA;
  CUtensorMap tm[2];
  int64_t blocks = 0;
  for (int i = 0; i < 2; ++i) {
    const OuterSide &o = a.side[i];
    if (!encode_bf16(&tm[i], o.X, o.N, a.seg.T, 1, o.ldx, 0, kORows, 2))
      return FP8LA_ERR_CUDA;
    blocks += (o.N + kOCols - 1) / kOCols;
  }
  const int64_t n = a.seg.n;
  // Two CTAs fit on an SM at ranks up to 32, but one is counted: two lead to
  // smaller clusters, which most of the sizes tried do not like.  Measured, us for a
  // backward pass counting one / two: rank 32, 4096 x 8192 with 3 adapters 97.4 /
  // 99.8, 1024 x 4096 with 4 27.7 / 30.5, 4096 x 2048 with 8 43.3 / 44.7, 4096 x
  // 4096 with 4 58.7 / 57.5; rank 8, 2048 x 2048 with 8 23.1 / 24.2; rank 16, 4096
  // x 4096 with 2 55.3 / 50.0, 4096 x 8192 with 1 90.4 / 79.9.
  const int cluster =
      choose_cluster(blocks * n, (a.seg.T + kORows * n - 1) / (kORows * n), sms(), 6);
  return launch(kern, dim3(cluster, static_cast<unsigned>(blocks),
                           static_cast<unsigned>(n)),
                kOThreads, C::kAlloc, cluster, s, tm[0], tm[1], a, wait_timeout_ns());
}

}  // namespace

fp8la_status launch_shrink_tma(const ShrinkArgs &a, cudaStream_t s) {
  return a.R <= 16   ? shrink_one<16>(a, 54, s)
         : a.R <= 32 ? shrink_one<32>(a, 55, s)
         : a.R <= 64 ? shrink_one<64>(a, 56, s)
                     : shrink_one<128>(a, 57, s);
}

fp8la_status launch_shrink_f32(const ShrinkArgs &a, cudaStream_t s) {
  return a.R <= 16   ? shrink_f32_one<16>(a, 65, s)
         : a.R <= 32 ? shrink_f32_one<32>(a, 66, s)
         : a.R <= 64 ? shrink_f32_one<64>(a, 67, s)
                     : shrink_f32_one<128>(a, 68, s);
}

fp8la_status launch_expand_tma(const ExpandArgs &a, cudaStream_t s) {
  return a.R <= 32 ? expand_one<32>(a, 63, s) : expand_one<64>(a, 64, s);
}

fp8la_status launch_outer_tma(const OuterArgs &a, cudaStream_t s) {
  return a.R <= 16   ? outer_one<16>(a, 58, s)
         : a.R <= 32 ? outer_one<32>(a, 59, s)
         : a.R <= 64 ? outer_one<64>(a, 60, s)
                     : outer_one<128>(a, 61, s);
}

}  // namespace lora
}  // namespace fp8la

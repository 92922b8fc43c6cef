// experts.cuh -- ragged products grouped by expert over a stack of 4-bit packs
// on the 5th-generation tensor cores, and the MXFP4 Linear (one expert):
//   Y[i] = X[i] W_e^T   for offsets[e] <= i < offsets[e + 1]
//
// The weights are the M side of the MMA (128 rows of W_e), the rows of X its N
// side: the instruction's N is a run-time value, so that a tile takes the rows
// that an expert has (rounded up to 16) instead of padding them to a tile, and a
// few rows per expert cost a few columns of MMA.
//
// The packed weights are dequantized straight into tensor memory: a
// dequantizer thread owns one weight row (one TMEM lane), turns 64 codes into 32
// words of bf16 pairs in registers and stores them with one tcgen05.st; the MMA
// reads them as its A operand.  The dequantized weights never pass through
// shared memory.
//
// One CTA walks items (expert, row tile, 128 weight rows).  Roles:
//   warp 0       codes [128 x 256 k] by TMA into a ring of WS stages
//   warp 1       X boxes [XBOX rows x 64 k] by TMA into a ring of XS slots of SK
//                k-blocks (64 k) each
//   warp 2       TMEM allocation and the MMA issuer (a whole warp in step, one
//                elected lane issues: a lone lane's branch costs 46 clocks an
//                instruction against 9 measured here)
//   warp 3       the experts' row tiles, then the scales (SEG bytes a row at a time)
//                and zero points of the codes' rows by cp.async, two segments deep
//   warps 4-19   dequantizers: four groups of four warps, one 64-wide k-block of
//                every chunk of 256 k each, into 32 columns of tensor memory
//   warps 20-23  epilogue: tcgen05.ld, transpose in shared memory, store Y
// All waits are bounded; see warp_wait.
#pragma once

#include <cuda_fp16.h>

#include "gemm_tcgen05.cuh"
#include "gemv_mma.cuh"
#include "mxfp4.cuh"
#include "wq_common.cuh"

namespace wq {

constexpr int kMaxExperts = 1024;  // a CTA keeps the experts' row bounds in shared memory
constexpr int kExpThreads = 768;
constexpr int kExpChunk = 256;     // k per stage of codes (128 bytes a row)

struct ExpertArgs {
  CUtensorMap tmW;         // codes u8 [E * N, K / 2], box {128, 128}, 128B swizzle
  CUtensorMap tmX;         // X bf16 [T, K], box {64, XBOX}, 128B swizzle
  const uint16_t* X;       // bf16 [T, K]
  const uint8_t* packed;   // K / 2 bytes per row, rows [E * N]
  const int* offsets;      // [E + 1], or null: one expert over all T rows
  const float* inv_s;      // fp32 [K] or null: multiplies column k of X (MXFP4 Linear)
  const uint16_t* scales;  // INT4 fp16 [E * N, K / G]
  const uint32_t* zeros;   // INT4 [E * N, ceil(K / G / 8)] or null (symmetric, z = 8)
  const uint8_t* bscale;   // NVFP4 E4M3 [E * N, K / 16]; MXFP4 E8M0 [E * N, K / 32]
  const float* gscale;     // NVFP4 fp32 [E]
  uint16_t* Y;             // bf16 [T, N]
  int E, N, K, T;
  int log2g;
  int split;               // CTAs of a cluster that share an item along K (1: none)
};

constexpr int kExpGroups = 4;      // dequantizer groups: one k-block of a chunk each

// Row bounds and first row tiles (of xt rows) of the experts, by one warp: bound[E + 1],
// tstart[E + 1], *bad = offsets that decrease or leave [0, T] (then nothing is computed).
__device__ __forceinline__ void expert_tables(const ExpertArgs& a, int xt, int* bound, int* tstart, int* bad_flag) {
  const int lane = threadIdx.x & 31;
  // each lane takes `per` experts in a row
  const int per = (a.E + 31) >> 5, e0 = min(a.E, lane * per), e1 = min(a.E, e0 + per);
  const auto bound_of = [&](int e) { return a.offsets ? __ldg(a.offsets + e) : (e ? a.T : 0); };
  bool bad = false;
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    const int b0 = bound_of(e), b1 = bound_of(e + 1);
    bad |= b0 < 0 || b1 < b0 || b1 > a.T;
    sum += bad ? 0 : (b1 - b0 + xt - 1) / xt;
  }
  bad = __any_sync(0xffffffffu, bad);
  int t = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, t, off);
    if (lane >= off) t += v;
  }
  t -= sum;
  for (int e = e0; e < e1; ++e) {
    const int b0 = bound_of(e), b1 = bound_of(e + 1);
    bound[e] = b0;
    tstart[e] = t;
    t += bad ? 0 : (b1 - b0 + xt - 1) / xt;
    if (e == a.E - 1) {
      bound[a.E] = b1;
      tstart[a.E] = t;
    }
  }
  if (lane == 0) {
    *bad_flag = bad;
    if (bad && blockIdx.x == 0) report_error(ERR_OFFSETS);
  }
}

// The last e with tstart[e] <= tile: the expert of a row tile.
__device__ __forceinline__ int expert_of_tile(const int* tstart, int E, int tile) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tstart[mid] <= tile) lo = mid; else hi = mid;
  }
  return lo;
}

// Up to XT rows of X per item, in boxes of XBOX; NACC accumulators (2: the
// epilogue overlaps the next item); WS stages of codes.  X slots and stages of
// dequantized weights hold SK k-blocks each: one pair of waits and one commit of the
// MMA issuer (about 300 clocks) for 4 SK instructions of XT / 2 clocks at most.
//
// Scales are fetched for many chunks at once, SEG bytes a row, because a warp's copy
// of 4 bytes from each of 32 rows takes as long as one of 16 bytes (about 200 clocks,
// more than the chunk's products).
template <int XT_, int XBOX_, int NACC_, int WS_, int XS_, int SK_, int SEG_>
struct ExpShape {
  static constexpr int XT = XT_, XBOX = XBOX_, NACC = NACC_, WS = WS_, XS = XS_, SK = SK_, SEG = SEG_;
  static constexpr int AS = SK == 1 ? 4 : 2;  // stages of dequantized weights, 32 SK columns each
  static constexpr int CODE_BYTES = 128 * 128;
  static constexpr int SC_PITCH = SEG + 16;     // a row's scales of a segment (a word more where rows start inside one)
  static constexpr int Z_PITCH = SEG / 4 + 4;   // a row's zero points of a segment: SEG / 2 groups
  static constexpr int META_BYTES = 128 * (SC_PITCH + Z_PITCH);
  static constexpr int SLOT_BYTES = SK * XT * 128;
  static constexpr int OFF_X = WS * CODE_BYTES;
  static constexpr int OFF_META = OFF_X + XS * SLOT_BYTES;
  static constexpr int OFF_STAGE = OFF_META + 2 * META_BYTES;
  static constexpr int OFF_TAB = OFF_STAGE + 4 * 1024;
  static constexpr int OFF_BAR = OFF_TAB + 2 * (kMaxExperts + 4) * 4;
  static constexpr int NBAR = 2 * WS + 2 * XS + AS + 2 * NACC + 4;
  static constexpr int SMEM_BYTES = OFF_BAR + NBAR * 8 + 64 + 1024;
  static constexpr int A_COL = NACC * XT;
  static constexpr int USED_COLS = A_COL + AS * SK * 32;
  static constexpr int TMEM_COLS = USED_COLS <= 256 ? 256 : 512;
  static_assert(USED_COLS <= 512, "tensor memory columns");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
  static_assert(XT % 16 == 0 && XT <= 256 && XT % XBOX == 0 && XBOX % 8 == 0, "row tiles");
  static_assert(SEG == 32 || SEG == 64, "a chunk takes 4 to 16 bytes of scales");
  static_assert(4 % SK == 0 && XS >= AS, "a dequantizer waits for the stage AS back on the slots' barriers");
  static_assert(WS * CODE_BYTES + XS * SLOT_BYTES >= XT * 128 * 4, "a split item's fp32 partial fits the rings");
};
using ExpWide = ExpShape<192, 32, 2, 3, 3, 2, 32>;
using ExpNarrow = ExpShape<64, 8, 2, 5, 3, 4, 64>;

// D[tmem] (+)= A[tmem] * B[smem]^T, bf16 inputs, fp32 accumulator.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// mbar_wait for a converged warp, with one answer for all its lanes: true once the
// phase of the given parity is complete, false on a timeout or another warp's abort.
// The global timer, slow to read, is looked at once in a thousand polls.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned err_bit, volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++i) {
    if ((i & 1023u) == 0) {
      const uint64_t now = globaltimer_ns();
      bool stop = *abort != 0;
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitLimitNs) {
        report_error(err_bit);
        *abort = 1;
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
  return true;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Asynchronous copy of BYTES bytes, the first src_bytes from global memory and the rest zeros.
template <int BYTES>
__device__ __forceinline__ void cp_async_zfill(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(src_bytes)
               : "memory");
}
// The barrier counts one arrival of this thread once its earlier cp.async have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One lane of a converged warp: the compiler then knows the branch's warp to be in step.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}

// d = a * b + c with fp16 a (half `hi_a` of a pair) and b, fp32 c and d.
template <int HI_A, int HI_B>
__device__ __forceinline__ float fma_f16_f32(uint32_t a, uint32_t b, float c) {
  float d;
  asm("{ .reg .b16 a0, a1, b0, b1;\n\t mov.b32 {a0, a1}, %1;\n\t mov.b32 {b0, b1}, %2;\n\t"
      "fma.rn.f32.f16 %0, a%4, b%5, %3; }"
      : "=f"(d)
      : "r"(a), "r"(b), "f"(c), "n"(HI_A), "n"(HI_B));
  return d;
}

// Dequantization is bound by the integer pipe (shifts, masks, permutes and the
// conversions), which takes an instruction of a warp every second clock, as the
// multiply-add pipe does for packed and integer products but not for fp32 ones with
// fp16 factors (every clock).  Measured on the alternatives: 5 clocks a pair of INT4
// codes and 4.3 of E2M1 codes in this form, 6 each with packed bf16 arithmetic.
//
// INT4: 16 (q - z) s of the 8 codes of a word in natural order, rounded to bf16 once:
// a code at bits 4-7 under the exponent of 1024 is the fp16 value 1024 + 16 q, and one
// multiply-add by the fp16 scale with c = -16 (64 + z) s (exact: 7 by 11 bits) gives
// 16 (q - z) s exactly in fp32.  The epilogue divides by 16.
__device__ __forceinline__ void dequant8_int4(uint32_t w, uint32_t s, float c, uint32_t* out) {
  constexpr uint32_t M = 0x00F000F0u, B = 0x64006400u;
  const uint32_t p0 = lop3_andor(w * 16u, M, B), p1 = lop3_andor(w, M, B);  // {code i, code i + 4}
  const uint32_t p2 = lop3_andor(w >> 4, M, B), p3 = lop3_andor(w >> 8, M, B);
  out[0] = pack_bf16x2(fma_f16_f32<0, 0>(p0, s, c), fma_f16_f32<0, 0>(p1, s, c));
  out[1] = pack_bf16x2(fma_f16_f32<0, 0>(p2, s, c), fma_f16_f32<0, 0>(p3, s, c));
  out[2] = pack_bf16x2(fma_f16_f32<1, 0>(p0, s, c), fma_f16_f32<1, 0>(p1, s, c));
  out[3] = pack_bf16x2(fma_f16_f32<1, 0>(p2, s, c), fma_f16_f32<1, 0>(p3, s, c));
}

// Byte B of w: two E2M1 codes as fp16 values, the first in the low half.
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_of_byte(uint32_t w) {
  uint32_t h;
  asm("{ .reg .b8 q0, q1, q2, q3;\n\t mov.b32 {q0, q1, q2, q3}, %1;\n\t cvt.rn.f16x2.e2m1x2 %0, q%2; }"
      : "=r"(h) : "r"(w), "n"(B));
  return h;
}
// E2M1: the 8 codes of a word times the fp16 scale in half HI of s, as bf16 pairs (exact).
template <int HI>
__device__ __forceinline__ void dequant8_e2m1(uint32_t w, uint32_t s, uint32_t* out) {
  const uint32_t h[4] = {e2m1x2_of_byte<0>(w), e2m1x2_of_byte<1>(w), e2m1x2_of_byte<2>(w), e2m1x2_of_byte<3>(w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = pack_bf16x2(fma_f16_f32<0, HI>(h[i], s, 0.f), fma_f16_f32<1, HI>(h[i], s, 0.f));
}
// The same times an fp32 scale and, where given, fp32 factors f[0..7] (rounded to bf16 once).
__device__ __forceinline__ void dequant8_e2m1_f32(uint32_t w, float s, const float* __restrict__ f, uint32_t* out) {
  const uint32_t h[4] = {e2m1x2_of_byte<0>(w), e2m1x2_of_byte<1>(w), e2m1x2_of_byte<2>(w), e2m1x2_of_byte<3>(w)};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    x[2 * i] = v.x * s;
    x[2 * i + 1] = v.y * s;
  }
  if (f) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(f)), b = __ldg(reinterpret_cast<const float4*>(f) + 1);
    x[0] *= a.x; x[1] *= a.y; x[2] *= a.z; x[3] *= a.w;
    x[4] *= b.x; x[5] *= b.y; x[6] *= b.z; x[7] *= b.w;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
}

template <int FMT, typename S>
__global__ void __launch_bounds__(kExpThreads, 1) expert_gemm_kernel(const __grid_constant__ ExpertArgs a) {
  constexpr int XT = S::XT, WS = S::WS, XS = S::XS, NACC = S::NACC, SK = S::SK, AS = S::AS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  int* bound = reinterpret_cast<int*>(smem + S::OFF_TAB);  // [E + 1] rows of the experts
  int* tstart = bound + kMaxExperts + 4;                   // [E + 1] their first row tile
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
  uint64_t* wfull = bars;                 // codes landed
  uint64_t* wempty = wfull + WS;          // dequantizers are done with them
  uint64_t* xfull = wempty + WS;          // X boxes landed
  uint64_t* mdone = xfull + XS;           // MMAs of the k-block in this slot finished
  uint64_t* aready = mdone + XS;          // dequantized weights in tensor memory
  uint64_t* dfull = aready + AS;          // accumulator complete
  uint64_t* dempty = dfull + NACC;        // accumulator drained
  uint64_t* sfull = dempty + NACC;        // [2] a segment of scales landed
  uint64_t* sempty = sfull + 2;           // [2] dequantizers are done with it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* bad_flag = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (warp == 0) {
    // arrivals: one of a thread that copies or commits, one of each dequantizer or epilogue warp
    if (lane < WS) { mbar_init(&wfull[lane], 1); mbar_init(&wempty[lane], 4 * kExpGroups); }
    if (lane < XS) { mbar_init(&xfull[lane], 1); mbar_init(&mdone[lane], 1); }
    if (lane < AS) mbar_init(&aready[lane], 4 * SK);
    if (lane < NACC) { mbar_init(&dfull[lane], 1); mbar_init(&dempty[lane], 4); }
    if (lane < 2) { mbar_init(&sfull[lane], 32); mbar_init(&sempty[lane], 4 * kExpGroups); }
    fence_mbar_init();
    if (lane == 0) {
      *abort_flag = 0;
      prefetch_tmap(&a.tmW);
      prefetch_tmap(&a.tmX);
    }
  } else if (warp == 2) {
    tmem_alloc(tmem_slot, S::TMEM_COLS);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 3) {
    expert_tables(a, XT, bound, tstart, bad_flag);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int nblocks = (a.N + 127) >> 7;
  const int items = *bad_flag ? 0 : tstart[a.E] * nblocks;
  const int nchunks = (a.K + kExpChunk - 1) / kExpChunk;
  // this CTA's items, and its chunks of an item
  int rank = 0, c0 = 0, c1 = nchunks, first = blockIdx.x, step = gridDim.x;
  if (a.split > 1) {
    rank = int(cluster_ctarank());
    c0 = nchunks * rank / a.split;
    c1 = nchunks * (rank + 1) / a.split;
    first /= a.split;
    step /= a.split;
  }

  struct Item {
    int e, row, rows, n0;  // expert, first row of X and their number, first weight row
  };
  const auto item_of = [&](int id) {
    Item it;
    const int tt = id / nblocks;
    it.n0 = (id - tt * nblocks) * 128;
    const int lo = expert_of_tile(tstart, a.E, tt);
    it.e = lo;
    const int r = bound[lo + 1] - bound[lo], t = tstart[lo + 1] - tstart[lo];
    const int w = ((r + t - 1) / t + 15) & ~15;  // the expert's rows, evenly over its tiles
    it.row = bound[lo] + (tt - tstart[lo]) * w;
    it.rows = min(w, bound[lo + 1] - it.row);
    return it;
  };
  // stages of a chunk: whole ones, the k-blocks past K are zeros (of the codes, the scales and X)
  const auto stages_of = [&](int c) { return min(4 / SK, (a.K - c * kExpChunk + 64 * SK - 1) / (64 * SK)); };
  // a row's scale bytes, those of a chunk, and the alignment that all rows share
  const uint8_t* sc_base = FMT == GEMM_INT4 ? reinterpret_cast<const uint8_t*>(a.scales) : a.bscale;
  const int sc_stride = FMT == GEMM_INT4 ? (a.K >> a.log2g) * 2 : FMT == GEMM_NVFP4 ? a.K >> 4 : a.K >> 5;
  const int sc_want = FMT == GEMM_INT4 ? (kExpChunk >> a.log2g) * 2 : FMT == GEMM_NVFP4 ? 16 : 8;
  const int sc_align = (sc_stride & 15) == 0 ? 16 : (sc_stride & 3) == 0 ? 4 : 1;
  const int cps = S::SEG / sc_want;  // chunks of a segment

  if (warp == 0) {
    // ---------------------------------------------------------- codes
    int q = 0, s = 0;
    uint32_t par = 1;  // parity of the stage's last use (the first use waits for none)
    bool ok = true;
    for (int id = first; id < items && ok; id += step) {
      const Item it = item_of(id);
      const int row0 = it.e * a.N + it.n0;
      for (int c = c0; c < c1; ++c, ++q) {
        if (q >= WS) ok = warp_wait(&wempty[s], par, ERR_TIMEOUT_PIPE, abort_flag);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&wfull[s], uint32_t(S::CODE_BYTES));
          tma_load_2d(smem + s * S::CODE_BYTES, &a.tmW, &wfull[s], c * 128, row0);
        }
        __syncwarp();
        if (++s == WS) {
          s = 0;
          par ^= 1u;
        }
      }
    }
    if (!ok) {  // let copies already issued land before the CTA leaves
      for (int k = (q > WS ? q - WS : 0); k < q; ++k) mbar_wait(&wfull[k % WS], (k / WS) & 1, ERR_TIMEOUT_TMA, nullptr);
    }
  } else if (warp == 3) {
    // ---------------------------------------------------------- scales and zero points
    int q = 0;
    bool ok = true;
    const int zw = ((a.K >> a.log2g) + 7) >> 3;
    for (int id = first; id < items && ok; id += step) {
      const Item it = item_of(id);
      const int64_t row0 = int64_t(it.e) * a.N + it.n0;
      const int valid = min(128, a.N - it.n0);  // rows past N get zeros
      for (int c = c0; c < c1; c = (c / cps + 1) * cps, ++q) {
        const int s = q & 1;
        if (q >= 2) ok = warp_wait(&sempty[s], ((q >> 1) - 1) & 1, ERR_TIMEOUT_PIPE, abort_flag);
        if (!ok) break;
        const uint32_t meta = sbase + uint32_t(S::OFF_META + s * S::META_BYTES);
        const int at = (c / cps) * S::SEG;                 // first byte of the segment within a row
        const int have = min(S::SEG, sc_stride - at);      // bytes past the row's end arrive as zeros
        if (sc_align == 16) {
          constexpr int PR = S::SEG / 16;                  // 16-byte pieces a row
          const int b = (lane % PR) * 16, n = max(0, min(16, have - b));
          const uint8_t* p = sc_base + (row0 + lane / PR) * sc_stride + at + b;
          uint32_t dst = meta + uint32_t((lane / PR) * S::SC_PITCH + b);
#pragma unroll 4
          for (int r = lane / PR; r < 128; r += 32 / PR, p += int64_t(32 / PR) * sc_stride, dst += 32 / PR * S::SC_PITCH) {
            const bool in = r < valid && n > 0;
            cp_async_zfill<16>(dst, in ? p : sc_base, in ? uint32_t(n) : 0u);
          }
        } else {
          // words; rows that start inside one: the words around the bytes, which the dequantizer shifts
          constexpr int PR = S::SEG / 4;
          const int b = (lane % PR) * 4;
          const uint8_t* p = sc_base + (row0 + lane / PR) * sc_stride + at;
          uint32_t dst = meta + uint32_t((lane / PR) * S::SC_PITCH + b);
#pragma unroll 4
          for (int r = lane / PR; r < 128; r += 32 / PR, p += int64_t(32 / PR) * sc_stride, dst += 32 / PR * S::SC_PITCH) {
            const int off = int(reinterpret_cast<uintptr_t>(p) & 3), n = max(0, min(4, off + have - b));
            const bool in = r < valid && n > 0;
            cp_async_zfill<4>(dst, in ? p - off + b : sc_base, in ? uint32_t(n) : 0u);
          }
          if (sc_align < 4) {
            for (int r = lane; r < 128; r += 32) {
              const uint8_t* e = sc_base + (row0 + r) * sc_stride + at;
              const int off = int(reinterpret_cast<uintptr_t>(e) & 3), n = max(0, min(4, off + have - S::SEG));
              const bool in = r < valid && n > 0;
              cp_async_zfill<4>(meta + uint32_t(r * S::SC_PITCH + S::SEG), in ? e - off + S::SEG : sc_base,
                                in ? uint32_t(n) : 0u);
            }
          }
        }
        if (FMT == GEMM_INT4 && a.zeros) {
          constexpr int PR = S::SEG / 16;  // words of eight zero points a row
          const int b = lane % PR, word = (c / cps) * PR + b;
#pragma unroll 4
          for (int r = lane / PR; r < 128; r += 32 / PR) {
            const bool in = r < valid && word < zw;
            cp_async_zfill<4>(meta + uint32_t(128 * S::SC_PITCH + r * S::Z_PITCH + b * 4),
                              in ? a.zeros + (row0 + r) * zw + word : reinterpret_cast<const uint32_t*>(sc_base),
                              in ? 4u : 0u);
          }
        }
        cp_async_arrive(&sfull[s]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 1) {
    // ---------------------------------------------------------- rows of X
    int q = 0, s = 0;
    uint32_t par = 1;
    bool ok = true;
    for (int id = first; id < items && ok; id += step) {
      const Item it = item_of(id);
      const int boxes = (it.rows + S::XBOX - 1) / S::XBOX;
      for (int c = c0; c < c1 && ok; ++c) {
        const int nst = stages_of(c);
        for (int h = 0; h < nst; ++h, ++q) {
          if (q >= XS) ok = warp_wait(&mdone[s], par, ERR_TIMEOUT_PIPE, abort_flag);
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&xfull[s], uint32_t(SK * boxes * S::XBOX) * 128u);
#pragma unroll
            for (int j = 0; j < SK; ++j)
              for (int b = 0; b < boxes; ++b)
                tma_load_2d(smem + S::OFF_X + s * S::SLOT_BYTES + j * XT * 128 + b * S::XBOX * 128, &a.tmX, &xfull[s],
                            c * kExpChunk + (h * SK + j) * 64, it.row + b * S::XBOX);
          }
          __syncwarp();
          if (++s == XS) {
            s = 0;
            par ^= 1u;
          }
        }
      }
    }
    if (!ok) {
      for (int k = (q > XS ? q - XS : 0); k < q; ++k) mbar_wait(&xfull[k % XS], (k / XS) & 1, ERR_TIMEOUT_TMA, nullptr);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------- MMA issuer
    int q = 0, i = 0, xs = 0, as = 0;
    uint32_t xpar = 0, apar = 0;
    bool ok = true;
    const uint64_t xd0 = desc_kmajor_sw128(sbase + uint32_t(S::OFF_X));
    for (int id = first; id < items && ok; id += step, ++i) {
      const Item it = item_of(id);
      const uint32_t idesc = idesc_bf16_f32(128, (it.rows + 15) & ~15);
      const int b = i % NACC, u = i / NACC;
      if (u > 0) ok = warp_wait(&dempty[b], (u - 1) & 1, ERR_TIMEOUT_PIPE, abort_flag);
      if (!ok) break;
      const uint32_t acc = tmem + uint32_t(b * XT);
      uint32_t more = 0;
      for (int c = c0; c < c1 && ok; ++c) {
        const int nst = stages_of(c);
        for (int h = 0; h < nst; ++h, ++q) {
          // both polled at once: in the steady state both are complete
          const bool xr = mbar_try_wait(&xfull[xs], xpar), ar = mbar_try_wait(&aready[as], apar);
          if (!__all_sync(0xffffffffu, xr && ar))
            ok = warp_wait(&xfull[xs], xpar, ERR_TIMEOUT_TMA, abort_flag) &&
                 warp_wait(&aready[as], apar, ERR_TIMEOUT_PIPE, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t xd = xd0 + uint64_t(uint32_t(xs * (S::SLOT_BYTES >> 4)));
            const uint32_t at = tmem + uint32_t(S::A_COL + as * SK * 32);
#pragma unroll
            for (int k = 0; k < 4 * SK; ++k)  // K = 16: 8 columns of A, 32 bytes inside X's swizzle atom
              umma_bf16_ts(acc, at + uint32_t(8 * k), xd + uint64_t((k >> 2) * (XT * 8) + 2 * (k & 3)), idesc,
                           more | uint32_t(k));
            umma_commit(&mdone[xs]);
          }
          __syncwarp();
          more = 1;
          if (++xs == XS) {
            xs = 0;
            xpar ^= 1u;
          }
          if (++as == AS) {
            as = 0;
            apar ^= 1u;
          }
        }
      }
      if (elect_one()) umma_commit(&dfull[b]);  // also after an abort: completes when the issued MMAs are done
      __syncwarp();
    }
  } else if (warp >= 4 && warp < 4 + 4 * kExpGroups) {
    // ---------------------------------------------------------- dequantizers
    const int kb = (warp - 4) >> 2;        // this group's k-block of every chunk
    const int quarter = warp & 3;          // TMEM lanes of this warp
    const int trow = quarter * 32 + lane;  // weight row within the tile
    const uint32_t a_tmem = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(S::A_COL + (kb % SK) * 32);
    const uint32_t my_codes = sbase + uint32_t(trow * 128);
    const uint32_t my_scales = sbase + uint32_t(S::OFF_META + trow * S::SC_PITCH);
    const uint32_t my_zeros = sbase + uint32_t(S::OFF_META + 128 * S::SC_PITCH + trow * S::Z_PITCH);
    // 16-byte pieces of this group's 32 bytes of a row, at their 128B-swizzled places
    const uint32_t piece0 = uint32_t(((2 * kb) ^ (trow & 7)) << 4), piece1 = uint32_t(((2 * kb + 1) ^ (trow & 7)) << 4);
    // byte within a row's chunk where this k-block's scales start
    const int sc_at = FMT == GEMM_INT4 ? ((kb * 64) >> a.log2g) * 2 : FMT == GEMM_NVFP4 ? 4 * kb : 2 * kb;
    int s = 0, as = 0, ms = 0;  // stage of the codes; stage of dequantized weights; slot whose MMAs free it
    int sg = 0;                 // segments of scales so far
    uint32_t wpar = 0, mpar = 0;
    int q = kb / SK;            // this group's stage number; the first AS stages are free from the start
    bool ok = true;
    as = q % AS;
    for (int id = first; id < items && ok; id += step) {
      const Item it = item_of(id);
      // row of the weights (mod 2^32: only its bytes' place within a word is asked for)
      const uint32_t srow = uint32_t(it.e) * uint32_t(a.N) + uint32_t(min(it.n0 + trow, a.N - 1));
      for (int c = c0, cs = c0 % cps; c < c1; ++c) {  // cs: chunk within its segment
        const int nst = stages_of(c);
        if (c == c0 || cs == 0) ok = warp_wait(&sfull[sg & 1], (sg >> 1) & 1, ERR_TIMEOUT_PIPE, abort_flag);
        ok = ok && warp_wait(&wfull[s], wpar, ERR_TIMEOUT_TMA, abort_flag);
        if (!ok) break;
        uint32_t v[32];
        if (kb < nst * SK) {
          const uint4 w0 = ld_shared_v4(my_codes + uint32_t(s * S::CODE_BYTES) + piece0);
          const uint4 w1 = ld_shared_v4(my_codes + uint32_t(s * S::CODE_BYTES) + piece1);
          const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
          const uint32_t meta = my_scales + uint32_t((sg & 1) * S::META_BYTES);
          int at = cs * sc_want + sc_at;  // this k-block's scales within the segment
          uint32_t sc;
          if (sc_align >= 4) {
            sc = ld_shared_u32(meta + uint32_t(at & ~3)) >> (8 * (at & 3));
          } else {  // the row starts inside a word (segments are whole words): four bytes from any place
            at += int((srow * uint32_t(sc_stride)) & 3u);
            sc = __funnelshift_r(ld_shared_u32(meta + uint32_t(at & ~3)), ld_shared_u32(meta + uint32_t((at & ~3) + 4)),
                                 8 * (at & 3));
          }
          if (FMT == GEMM_INT4) {
            uint32_t zword = 0x88888888u;
            const int g = (cs * kExpChunk + kb * 64) >> a.log2g;  // the k-block's first group within the segment
            if (a.zeros) zword = ld_shared_u32(my_zeros + uint32_t((sg & 1) * S::META_BYTES + (g >> 3) * 4));
            zword >>= 4 * (g & 7);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bool second = h == 1 && a.log2g == 5;  // G = 32: two groups in the k-block
              const uint32_t s16 = second ? sc >> 16 : sc;
              const float z = float((second ? zword >> 4 : zword) & 15u);
              const float cz = -16.f * (64.f + z) * __half2float(__ushort_as_half(uint16_t(s16)));
#pragma unroll
              for (int j = 0; j < 4; ++j) dequant8_int4(w[4 * h + j], s16, cz, v + 16 * h + 4 * j);
            }
          } else if (FMT == GEMM_NVFP4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t s2;  // the scales of the two blocks, fp16 (exact)
              asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }"
                  : "=r"(s2) : "r"((sc >> (16 * h)) & 0x7F7Fu));
              dequant8_e2m1<0>(w[4 * h], s2, v + 16 * h);
              dequant8_e2m1<0>(w[4 * h + 1], s2, v + 16 * h + 4);
              dequant8_e2m1<1>(w[4 * h + 2], s2, v + 16 * h + 8);
              dequant8_e2m1<1>(w[4 * h + 3], s2, v + 16 * h + 12);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t e8 = (sc >> (8 * h)) & 255u;
              // a scale that is a normal fp16 (2^-14 .. 2^15) for the whole warp, or fp32 products
              if (!a.inv_s && __all_sync(0xffffffffu, e8 - 113u < 30u)) {
                const uint32_t s2 = (e8 - 112u) << 10;
#pragma unroll
                for (int j = 0; j < 4; ++j) dequant8_e2m1<0>(w[4 * h + j], s2, v + 16 * h + 4 * j);
              } else {
                const int k0 = c * kExpChunk + kb * 64 + h * 32;
                const float* f = a.inv_s && k0 < a.K ? a.inv_s + k0 : nullptr;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  dequant8_e2m1_f32(w[4 * h + j], e8m0_f32(e8), f ? f + 8 * j : nullptr, v + 16 * h + 4 * j);
              }
            }
          }
          // the columns are free once the MMAs of the stage AS back are done
          if (q >= AS) {
            ok = warp_wait(&mdone[ms], mpar, ERR_TIMEOUT_PIPE, abort_flag);
            if (!ok) break;
          }
          tc_fence_after();
          tmem_st32(a_tmem + uint32_t(as * SK * 32), v);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) {
          if (kb < nst * SK) mbar_arrive(&aready[as]);
          mbar_arrive(&wempty[s]);
          if (cs == cps - 1 || c == c1 - 1) mbar_arrive(&sempty[sg & 1]);
        }
        if (++cs == cps) cs = 0;
        if (cs == 0 || c == c1 - 1) ++sg;
        // stages up to this group's place in the next chunk
        for (int j = 0; j < nst; ++j) {
          if (++as == AS) as = 0;
          if (q++ >= AS && ++ms == XS) {
            ms = 0;
            mpar ^= 1u;
          }
        }
        if (++s == WS) {
          s = 0;
          wpar ^= 1u;
        }
      }
    }
  } else if (warp >= 4 + 4 * kExpGroups) {
    // ---------------------------------------------------------- epilogue
    const int quarter = warp & 3;
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    const bool vec = (a.N & 7) == 0;
    uint8_t* stage = smem + S::OFF_STAGE + quarter * 1024;  // 16 rows of X x 32 weight rows, bf16
    int i = 0;
    for (int id = first; id < items; id += step, ++i) {
      const Item it = item_of(id);
      const int b = i % NACC, u = i / NACC;
      const float gmul = FMT == GEMM_NVFP4 ? __ldg(a.gscale + it.e) : FMT == GEMM_INT4 ? 0.0625f : 1.0f;
      if (!warp_wait(&dfull[b], u & 1, ERR_TIMEOUT_MMA, abort_flag)) break;
      tc_fence_after();
      const int nw = it.n0 + quarter * 32;  // this warp's first weight row
      for (int x = 0; x < it.rows; x += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + lane_base + uint32_t(b * XT + x), v);
        if (a.split > 1) {
          // this CTA's part of the sums, fp32 [rows][128] over the rings (every copy and MMA
          // of this only item is done)
          float* part = reinterpret_cast<float*>(smem);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (x + j < it.rows) part[(x + j) * 128 + quarter * 32 + lane] = __uint_as_float(v[j]) * gmul;
          continue;
        }
        if (!vec) {
          const int n = nw + lane;
          if (n < a.N) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (x + j < it.rows) {
                const float y = __uint_as_float(v[j]) * gmul;
                a.Y[int64_t(it.row + x + j) * a.N + n] = uint16_t(pack_bf16x2(y, y));
              }
          }
          continue;
        }
#pragma unroll
        for (int h = 0; h < 32; h += 16) {  // 16 rows of X: transpose, then 16-byte pieces of Y's rows
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const uint32_t y2 = pack_bf16x2(__uint_as_float(v[h + j]) * gmul, __uint_as_float(v[h + j + 1]) * gmul);
            *reinterpret_cast<uint16_t*>(stage + j * 64 + lane * 2) = uint16_t(y2);
            *reinterpret_cast<uint16_t*>(stage + (j + 1) * 64 + lane * 2) = uint16_t(y2 >> 16);
          }
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 16; p += 8) {
            const int j = p + (lane >> 2), n = nw + (lane & 3) * 8;
            if (x + h + j < it.rows && n < a.N)
              *reinterpret_cast<uint4*>(a.Y + int64_t(it.row + x + h + j) * a.N + n) =
                  *reinterpret_cast<const uint4*>(stage + j * 64 + (lane & 3) * 16);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&dempty[b]);
    }
  }
  __syncwarp();
  if (a.split > 1 && first < items) {
    // one item per cluster: rank r adds rows r, r + split, .. over the ranks' parts, in rank order
    cluster_sync();
    const Item it = item_of(first);
    const int n = it.n0 + (threadIdx.x & 127);
    if (!*abort_flag && n < a.N) {
      for (int x = rank + a.split * (threadIdx.x >> 7); x < it.rows; x += a.split * (kExpThreads / 128)) {
        const uint32_t at = sbase + uint32_t(x * 128 + (threadIdx.x & 127)) * 4u;
        float p[8], y = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) p[r] = r < a.split ? ld_shared_cluster_f32(map_shared_rank(at, uint32_t(r))) : 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) y += p[r];
        a.Y[int64_t(it.row + x) * a.N + n] = uint16_t(pack_bf16x2(y, y));
      }
    }
    cluster_sync();  // the parts stay until every rank has read them
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, S::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// Few rows per expert: mma.sync with the weights (16 rows of W_e) as the A operand,
// dequantized in registers, and up to 8 NT rows of X as B.  Bound by HBM (0.53 to
// 0.63 bytes a weight) and by the dequantization's instructions, both within 20%.
//
// A unit is 16 weight rows of one row tile; its steps are 128 k each.  A CTA takes a
// contiguous share of the units, its warps contiguous shares of the CTA's steps, so that
// every SM streams the same number of bytes whatever K is, and only units that
// straddle warps are summed through shared memory, in warp order.  A step's codes come
// by cp.async, kVecDepth steps ahead, into slots that the copying lane reads itself
// (no barrier, and a loop body of one step: the kernel is short, and a body unrolled
// over the steps in flight spent most of it on instruction fetches); scales and a
// word's rows of X one step ahead into registers (L2 holds the scales' sector from the
// first step that touched it, L1 the rows that all warps of a CTA read).
// Lane (g, c) (g = lane / 4, c = lane % 4) holds codes of rows g and g + 8: the k order
// inside an MMA is free, so its four k of each are four consecutive k of the lane's.
//   INT4   lane c takes G / 4 k of every group, so that an MMA stays inside a group: A is
//          q - z (exact in bf16), and the fp16 scale multiplies the group's fp32 sums;
//   E2M1   lane c takes 32 k in a row; A is the code times its block scale, exact in bf16.
constexpr int kVecWarps = 16;
constexpr int kVecDepth = 4;
constexpr int kVecSmem = kVecWarps * kVecDepth * 1024;

// FULL: K % 128 == 0, no step reaches past K (and scale bytes of a step are aligned words).
__device__ __forceinline__ uint32_t ldg_u16(const void* p) { return __ldg(static_cast<const uint16_t*>(p)); }
__device__ __forceinline__ uint32_t ldg_u8(const void* p) { return __ldg(static_cast<const uint8_t*>(p)); }

template <int FMT, int G, int NT, bool FULL>
__global__ void __launch_bounds__(kVecWarps * 32, 1) expert_gemv_kernel(const __grid_constant__ ExpertArgs a) {
  static_assert(FMT != GEMM_INT4 || G == 32 || G == 64 || G == 128, "group size");
  constexpr int NG = FMT == GEMM_INT4 ? 128 / G : 1;    // groups of a step
  constexpr int WPG = 4 / NG;                           // words (8 k) of a lane per group
  __shared__ int bound[kMaxExperts + 4], tstart[kMaxExperts + 4];
  __shared__ int bad_flag;
  __shared__ float part[2 * kVecWarps][16][8 * NT];     // sums of units that straddle warps
  extern __shared__ __align__(16) uint8_t vec_smem[];   // codes: [warp][kVecDepth][2][32 lanes][16 bytes]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int K = a.K, N = a.N;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 0) expert_tables(a, 8 * NT, bound, tstart, &bad_flag);
  __syncthreads();
  if (bad_flag) return;
  const int nrb = (N + 15) >> 4, S = (K + 127) >> 7;  // row blocks of an expert, steps of a unit
  // the CTA's units and the warps' first steps of them
  const int units = tstart[a.E] * nrb, per = units / gridDim.x, more = units - per * gridDim.x;
  const int u0 = blockIdx.x * per + min(int(blockIdx.x), more), nu = per + (int(blockIdx.x) < more);
  const int tot = nu * S;
  const auto first_of = [&](int w) { return int(int64_t(tot) * w / kVecWarps); };

  struct Unit {
    int e, row, rows, n0;
  };
  const auto unit_of = [&](int u) {
    Unit t;
    const int tile = u / nrb;
    t.n0 = (u - tile * nrb) * 16;
    t.e = expert_of_tile(tstart, a.E, tile);
    const int r = bound[t.e + 1] - bound[t.e], nt = tstart[t.e + 1] - tstart[t.e];
    const int w = (r + nt - 1) / nt;  // the expert's rows, evenly over its tiles
    t.row = bound[t.e] + (tile - tstart[t.e]) * w;
    t.rows = min(w, bound[t.e + 1] - t.row);
    return t;
  };
  // k of word j (8 codes) of this lane within a step
  const auto k_of = [&](int j) { return FMT == GEMM_INT4 ? (j / WPG) * G + c * (G / 4) + (j % WPG) * 8 : 32 * c + 8 * j; };
  const int zw = (((FMT == GEMM_INT4 ? K / G : 8) + 7) >> 3) * 4;  // zero-point bytes of a row
  const int sw = FMT == GEMM_INT4 ? K / G * 2 : FMT == GEMM_NVFP4 ? K >> 4 : K >> 5;  // scale bytes of a row
  const uint8_t* sbase = FMT == GEMM_INT4 ? reinterpret_cast<const uint8_t*>(a.scales) : a.bscale;

  const uint32_t ring = smem_u32(vec_smem) + uint32_t(warp * kVecDepth * 1024 + lane * 16);
  int at = first_of(warp);
  const int end = first_of(warp + 1);
  while (at < end) {
    // ---- the warp's steps [ja, jb) of a unit
    const int u = at / S, ja = at - u * S, jb = min(S, ja + end - at);
    at += jb - ja;
    const Unit t = unit_of(u0 + u);
    const int64_t rlo = int64_t(t.e) * N + min(t.n0 + g, N - 1), rhi = int64_t(t.e) * N + min(t.n0 + g + 8, N - 1);
    // cursors: codes kVecDepth - 1 steps ahead, scales and X one step ahead
    const uint8_t* plo = a.packed + rlo * (K >> 1) + ja * 64 + (FMT == GEMM_INT4 ? c * (G / 8) : 16 * c);
    const uint8_t* phi = plo + (rhi - rlo) * (K >> 1);
    constexpr int SB = FMT == GEMM_INT4 ? 2 * NG : FMT == GEMM_NVFP4 ? 8 : 4;  // scale bytes of a step
    const uint8_t* slo = sbase + rlo * sw + ja * SB + (FMT == GEMM_NVFP4 ? 2 * c : FMT == GEMM_MXFP4 ? c : 0);
    const uint8_t* shi = slo + (rhi - rlo) * sw;
    const uint8_t* zlo = reinterpret_cast<const uint8_t*>(a.zeros) + rlo * zw;
    const uint8_t* zhi = zlo + (rhi - rlo) * zw;
    const uint16_t* xp[NT];  // this lane's rows of X; a lane without one reads the tile's last (its sums are not stored)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      xp[n] = a.X + int64_t(t.row + min(8 * n + g, t.rows - 1)) * K + ja * 128 + (FMT == GEMM_INT4 ? c * (G / 4) : 32 * c);

    // a lane's 16 code bytes of each row, in word order; zeros past K
    uint32_t put = ring + uint32_t(ja % kVecDepth) * 1024u;
    const auto request = [&](int j) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const bool in = FULL || (FMT == GEMM_INT4 ? j * 128 + i * G < K : j * 128 + 32 * c < K);
        cp_async_zfill<16 / NG>(put + i * (16 / NG), in ? plo + i * (G / 2) : a.packed, in ? 16 / NG : 0);
        cp_async_zfill<16 / NG>(put + 512 + i * (16 / NG), in ? phi + i * (G / 2) : a.packed, in ? 16 / NG : 0);
      }
      plo += 64;
      phi += 64;
      put = put + 1024u == ring + kVecDepth * 1024u ? ring : put + 1024u;
    };
    // scales, row g's in the low half (fp16 per group, two E4M3 bytes, or an E8M0 byte), and
    // the bytes that hold the step's zero points (one for G >= 64, else two)
    uint32_t sc[NG], zp = 0x88888888u;
    const auto load_scales = [&](int j) {
      if (FMT == GEMM_INT4 && FULL && NG > 1) {  // a row's scales of the step as words
#pragma unroll
        for (int i = 0; i < NG; i += 2) {
          const uint32_t l = __ldg(reinterpret_cast<const uint32_t*>(slo + 2 * i));
          const uint32_t h = __ldg(reinterpret_cast<const uint32_t*>(shi + 2 * i));
          sc[i] = prmt_b32(l, h, 0x5410);
          sc[(i + 1) % NG] = prmt_b32(l, h, 0x7632);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const bool in = FULL || (FMT == GEMM_INT4 ? (j * NG + i) * 2 < sw : j * 128 + 32 * c < K);
          sc[i] = !in ? 0u : FMT == GEMM_MXFP4 ? ldg_u8(slo) | (ldg_u8(shi) << 16)
                                               : ldg_u16(slo + 2 * i) | (ldg_u16(shi + 2 * i) << 16);
        }
      }
      slo += SB;
      shi += SB;
      if (FMT == GEMM_INT4 && a.zeros) {
        const int b = (j * NG) >> 1;
        zp = G == 32 ? ldg_u16(zlo + b) | (ldg_u16(zhi + b) << 16) : ldg_u8(zlo + b) | (ldg_u8(zhi + b) << 16);
      }
    };
    const auto xload = [&](int n, int w, int j) {
      const int k = FMT == GEMM_INT4 ? (w / WPG) * G + (w % WPG) * 8 : 8 * w;  // past the lane's first of the step
      return FULL || j * 128 + k_of(w) < K ? ldg_v4(xp[n] + k) : make_uint4(0, 0, 0, 0);
    };

    uint4 x[NT][4];
    float acc[NT][4];
#pragma unroll 1
    for (int i = 0; i < kVecDepth - 1; ++i) {
      if (ja + i < jb) request(ja + i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    load_scales(ja);
    uint32_t take = ring + uint32_t(ja % kVecDepth) * 1024u;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int w = 0; w < 4; ++w) x[n][w] = xload(n, w, ja);
      xp[n] += 128;
      acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    }
#pragma unroll 1
    for (int j = ja; j < jb; ++j) {
      if (j + kVecDepth - 1 < jb) request(j + kVecDepth - 1);
      asm volatile("cp.async.commit_group;\n\tcp.async.wait_group %0;" ::"n"(kVecDepth - 1) : "memory");
      const uint4 cl = ld_shared_v4(take), ch = ld_shared_v4(take + 512);
      take = take + 1024u == ring + kVecDepth * 1024u ? ring : take + 1024u;
      const uint32_t wl[4] = {cl.x, cl.y, cl.z, cl.w}, wh[4] = {ch.x, ch.y, ch.z, ch.w};
      uint32_t s[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) s[i] = sc[i];
      const uint32_t z = zp;
      if (j + 1 < jb) load_scales(j + 1);
      uint32_t s2lo = 0, s2hi = 0;
      bool f16 = true;  // MXFP4: the warp's block scales are normal fp16 values
      if (FMT == GEMM_NVFP4) {
        s2lo = tc_e4m3x2(s[0] & 0x7F7Fu);
        s2hi = tc_e4m3x2((s[0] >> 16) & 0x7F7Fu);
      } else if (FMT == GEMM_MXFP4) {
        const uint32_t el = s[0] & 255u, eh = s[0] >> 16;
        f16 = __all_sync(0xffffffffu, el - 113u < 30u && eh - 113u < 30u);
        s2lo = f16 ? (el - 112u) << 10 : __float_as_uint(e8m0_f32(el));
        s2hi = f16 ? (eh - 112u) << 10 : __float_as_uint(e8m0_f32(eh));
      }
      float d[NT][4];  // INT4: the group's sums
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t al[4], ah[4];
        if (FMT == GEMM_INT4) {
          const int nib = 4 * ((G == 128 ? (j & 1) : 0) + w / WPG);  // this group's zero point
          const uint32_t zl = 0x43004300u + ((z >> nib) & 15u) * 0x00010001u;
          const uint32_t zh = 0x43004300u + ((z >> (16 + nib)) & 15u) * 0x00010001u;
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // {code q, code q + 4}
            al[q] = bf16x2_sub(lop3_andor(wl[w] >> (4 * q), 0x000F000Fu, 0x43004300u), zl);
            ah[q] = bf16x2_sub(lop3_andor(wh[w] >> (4 * q), 0x000F000Fu, 0x43004300u), zh);
          }
        } else if (FMT == GEMM_NVFP4) {
          if (w < 2) {
            dequant8_e2m1<0>(wl[w], s2lo, al);
            dequant8_e2m1<0>(wh[w], s2hi, ah);
          } else {
            dequant8_e2m1<1>(wl[w], s2lo, al);
            dequant8_e2m1<1>(wh[w], s2hi, ah);
          }
        } else if (f16) {
          dequant8_e2m1<0>(wl[w], s2lo, al);
          dequant8_e2m1<0>(wh[w], s2hi, ah);
        } else {
          dequant8_e2m1_f32(wl[w], __uint_as_float(s2lo), nullptr, al);
          dequant8_e2m1_f32(wh[w], __uint_as_float(s2hi), nullptr, ah);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 b = x[n][w];
          if (j + 1 < jb) x[n][w] = xload(n, w, j + 1);
          const int k = j * 128 + k_of(w);
          if (FMT == GEMM_MXFP4 && a.inv_s && k < K) {  // X * act_inv_s, rounded to bf16 once
            const float4 i0 = __ldg(reinterpret_cast<const float4*>(a.inv_s + k));
            const float4 i1 = __ldg(reinterpret_cast<const float4*>(a.inv_s + k) + 1);
            b.x = pack_bf16x2(__uint_as_float(b.x << 16) * i0.x, __uint_as_float(b.x & 0xFFFF0000u) * i0.y);
            b.y = pack_bf16x2(__uint_as_float(b.y << 16) * i0.z, __uint_as_float(b.y & 0xFFFF0000u) * i0.w);
            b.z = pack_bf16x2(__uint_as_float(b.z << 16) * i1.x, __uint_as_float(b.z & 0xFFFF0000u) * i1.y);
            b.w = pack_bf16x2(__uint_as_float(b.w << 16) * i1.z, __uint_as_float(b.w & 0xFFFF0000u) * i1.w);
          }
          if (FMT == GEMM_INT4) {
            if (w % WPG == 0) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
            // {x0, x4} {x1, x5} | {x2, x6} {x3, x7}
            mma_bf16_16816(d[n], al[0], ah[0], al[1], ah[1], prmt_b32(b.x, b.z, 0x5410), prmt_b32(b.x, b.z, 0x7632));
            mma_bf16_16816(d[n], al[2], ah[2], al[3], ah[3], prmt_b32(b.y, b.w, 0x5410), prmt_b32(b.y, b.w, 0x7632));
            if (w % WPG == WPG - 1) {
              const float sl = __half2float(__ushort_as_half(uint16_t(s[w / WPG])));
              const float sh = __half2float(__ushort_as_half(uint16_t(s[w / WPG] >> 16)));
              acc[n][0] = fmaf(sl, d[n][0], acc[n][0]);
              acc[n][1] = fmaf(sl, d[n][1], acc[n][1]);
              acc[n][2] = fmaf(sh, d[n][2], acc[n][2]);
              acc[n][3] = fmaf(sh, d[n][3], acc[n][3]);
            }
          } else {
            mma_bf16_16816(acc[n], al[0], ah[0], al[1], ah[1], b.x, b.y);
            mma_bf16_16816(acc[n], al[2], ah[2], al[3], ah[3], b.z, b.w);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) xp[n] += 128;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // ---- rows g and g + 8, columns 8 n + 2 c (+ 1): the unit's result, or the warp's share of it
    if (ja == 0 && jb == S) {
      const float gmul = FMT == GEMM_NVFP4 ? __ldg(a.gscale + t.e) : 1.f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int m = 8 * n + 2 * c + (q & 1), r = t.n0 + g + (q >> 1) * 8;
          const float y = acc[n][q] * gmul;
          if (m < t.rows && r < N) a.Y[int64_t(t.row + m) * N + r] = uint16_t(pack_bf16x2(y, y));
        }
    } else {
      // slot 2 w: the unit was begun by an earlier warp; 2 w + 1: a later one ends it
      float (*p)[8 * NT] = part[2 * warp + (ja == 0)];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) p[g + (q >> 1) * 8][8 * n + 2 * c + (q & 1)] = acc[n][q];
    }
  }
  __syncthreads();
  // ---- the warp that ends a unit begun by an earlier one adds the shares in warp order
  const int s0 = first_of(warp), u = s0 / S, ub = u * S;  // the unit of the warp's first step, and that unit's first
  if (s0 < end && s0 > ub && end >= ub + S) {
    int v = warp - 1;
    while (first_of(v) > ub) --v;
    const Unit t = unit_of(u0 + u);
    const float gmul = FMT == GEMM_NVFP4 ? __ldg(a.gscale + t.e) : 1.f;
    for (int i = lane; i < 16 * 8 * NT; i += 32) {
      const int r = i & 15, m = i >> 4;
      float y = 0.f;
      for (int w = v; w <= warp; ++w)
        if (first_of(w) < first_of(w + 1)) y += part[2 * w + (first_of(w) <= ub)][r][m];
      y *= gmul;
      if (m < t.rows && t.n0 + r < N) a.Y[int64_t(t.row + m) * N + t.n0 + r] = uint16_t(pack_bf16x2(y, y));
    }
  }
}

}  // namespace wq

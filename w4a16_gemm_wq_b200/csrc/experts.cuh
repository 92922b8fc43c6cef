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
//   warp 1       X boxes [rows x 64 k] by TMA into a ring of XS slots of SK
//                k-blocks (64 k) each
//   warp 2       TMEM allocation and the MMA issuer (a whole warp in step, one
//                elected lane issues: a lone lane's branch costs 46 clocks an
//                instruction against 9 measured here)
//   warp 3       the experts' row tiles, then the scales (SEG bytes a row at a time)
//                and zero points of the codes' rows by cp.async, two segments deep
//   warps 4-19   dequantizers: four groups of four warps, one 64-wide k-block of
//                every chunk of 256 k each, into 32 columns of tensor memory
//   warps 20-23  epilogue: tcgen05.ld, store Y
// All waits are bounded; see warp_wait.
//
// Bound by the MMAs where rows are many and by the conversions where they are few: an item's
// chunk of 256 k takes 8 clocks a row of X in the tensor pipe, and about 1900 clocks to
// convert and store, whatever its rows; what a chunk's four dequantizer warps of a scheduler
// wait for does not overlap (two chunks a wait, or the groups started apart, measured the same).
// 2048 x 11008 x 2048 MXFP4: 70.2 us, 1316 TFLOP/s (tensor pipe 70% busy, issue 65%; without
// conversions and their store 58.8 us); 16384 rows over 64 NVFP4 experts of 1408 x 2048: 94 us,
// 1002 TFLOP/s; 13 x 28672 x 4096: 36 us.
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
  CUtensorMap tmX[6];      // X bf16 [T, K], boxes {64, xunit * (1 .. xmaps)}, 128B swizzle
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
  int xunit, xmaps;        // heights of X's boxes
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

// Shape of the tcgen05 form: up to XT rows of X per item; NACC accumulators (2: the
// epilogue overlaps the next item); WS stages of codes.  X slots and stages of
// dequantized weights hold SK k-blocks each: one pair of waits and one commit of the
// MMA issuer (about 300 clocks) for 4 SK instructions of XT / 2 clocks at most.  The same
// shape serves few rows: an item's boxes and MMAs are as high as its rows (tiles of 64 rows
// with deeper stages were within 2% at 13 to 1000 rows, and slower from 64 an expert on; of
// 256 rows with one accumulator: 200 x 28672 x 4096 in 50 us against 66, but 100 rows of it
// in 42 against 38, and 48 rows for each of 64 experts in 55 against 48).
//
// Scales are fetched for many chunks at once, SEG bytes a row, because a warp's copy
// of 4 bytes from each of 32 rows takes as long as one of 16 bytes (about 200 clocks,
// more than the chunk's products).
//
// A k-block of X is one TMA box of the item's height, rounded up to XUNIT (a map for each):
// a box takes its thread about 100 clocks whatever its height, and six of 32 rows took
// longer than the k-block's products (2048 x 11008 x 2048: 76.7 -> 73.4 us).
struct ExpShape {
  static constexpr int XT = 192, XUNIT = 32, NACC = 2, WS = 3, XS = 3, SK = 2, SEG = 32;
  static constexpr int AS = 2;                  // stages of dequantized weights, 32 SK columns each
  static constexpr int CODE_BYTES = 128 * 128;
  static constexpr int SC_PITCH = SEG + 16;     // a row's scales of a segment (a word more where rows start inside one)
  static constexpr int Z_PITCH = SEG / 4 + 4;   // a row's zero points of a segment: SEG / 2 groups
  static constexpr int META_BYTES = 128 * (SC_PITCH + Z_PITCH);
  static constexpr int SLOT_BYTES = SK * XT * 128;
  static constexpr int OFF_X = WS * CODE_BYTES;
  static constexpr int OFF_META = OFF_X + XS * SLOT_BYTES;
  static constexpr int OFF_TAB = OFF_META + 2 * META_BYTES;
  static constexpr int OFF_BAR = OFF_TAB + 2 * (kMaxExperts + 4) * 4;
  static constexpr int NBAR = 2 * WS + 2 * XS + AS + 2 * NACC + 4;
  static constexpr int SMEM_BYTES = OFF_BAR + NBAR * 8 + 64 + 1024;
  static constexpr int A_COL = NACC * XT;       // tensor memory: accumulators, then dequantized weights
  static constexpr int TMEM_COLS = 512;
  static_assert(A_COL + AS * SK * 32 <= TMEM_COLS, "tensor memory columns");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
  static_assert(XT % XUNIT == 0 && XUNIT % 16 == 0, "row tiles");
  // A dequantizer waits for the stage AS back on the slots' barriers.  Where the last chunk of K has
  // no k-block for its group, its next stage is up to 8 / SK - 1 after its last: it must have seen the
  // slot's phase before the awaited one (of the stage XS earlier), which its parity alone could pass for.
  static_assert(XS >= AS && XS >= 8 / SK - 1, "phases that a dequantizer may miss");
  static_assert(WS * CODE_BYTES + XS * SLOT_BYTES >= XT * 128 * 4, "a split item's fp32 partial fits the rings");
};

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
// fp16 factors (every clock).  Measured, 16 warps, 64 codes a lane with their store: 1055
// clocks (INT4) and 843 (E2M1) in this form; 996 and 922 in packed bf16 arithmetic
// rounded once (INT4 without the split of its scale into two bf16), 322 the store alone.
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

// What the non-finite elements of a row of X make of its product with a weight row: an infinity,
// or NaN (0 for a row without any).  For the forms for few rows, whose own arithmetic takes away
// what it added (INT4) or multiplies blocks of another scale by zero (MXFP4): with an infinity
// both leave NaN where the product is one.  Read again from memory, by one thread: rare, and
// out of line for the registers and the length of what is not.
template <int FMT>
__device__ __noinline__ float nonfinite_terms(const ExpertArgs& a, int64_t xrow, int64_t wrow) {
  static_assert(FMT == GEMM_INT4 || FMT == GEMM_MXFP4, "NVFP4 needs none");
  float y = 0.f;
#pragma unroll 1
  for (int k = 0; k < a.K; ++k) {
    float x = bf16_bits_to_f32(a.X[xrow * a.K + k]);
    if (FMT == GEMM_MXFP4 && a.inv_s) x *= a.inv_s[k];
    if ((__float_as_uint(x) & 0x7FFFFFFFu) < 0x7F800000u) continue;
    const uint32_t code = (a.packed[wrow * (a.K >> 1) + (k >> 1)] >> (4 * (k & 1))) & 15u;
    if (FMT == GEMM_INT4) {
      const int ng = a.K >> a.log2g, g = k >> a.log2g;
      const uint32_t z = a.zeros ? (a.zeros[wrow * ((ng + 7) >> 3) + (g >> 3)] >> (4 * (g & 7))) & 15u : 8u;
      y += (float(code) - float(z)) * __half2float(__ushort_as_half(a.scales[wrow * ng + g])) * x;
    } else {
      const uint32_t h = e2m1x2_of_byte<0>(code);
      y += __half2float(__ushort_as_half(uint16_t(h))) * e8m0_f32(a.bscale[wrow * (a.K >> 5) + (k >> 5)]) * x;
    }
  }
  return y;
}

template <int FMT>
__global__ void __launch_bounds__(kExpThreads, 1) expert_gemm_kernel(const __grid_constant__ ExpertArgs a) {
  using S = ExpShape;
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
      for (int b = 0; b < a.xmaps; ++b) prefetch_tmap(&a.tmX[b]);
    }
  } else if (warp == 2) {
    tmem_alloc(tmem_slot, S::TMEM_COLS);
    tmem_relinquish();
  }
  // what needs no memory is computed while the kernel before this one ends
  const int nblocks = (a.N + 127) >> 7;
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
  // a row's scale bytes, those of a chunk, and the alignment that all rows share
  const uint8_t* sc_base = FMT == GEMM_INT4 ? reinterpret_cast<const uint8_t*>(a.scales) : a.bscale;
  const int sc_stride = FMT == GEMM_INT4 ? (a.K >> a.log2g) * 2 : FMT == GEMM_NVFP4 ? a.K >> 4 : a.K >> 5;
  const int sc_want = FMT == GEMM_INT4 ? (kExpChunk >> a.log2g) * 2 : FMT == GEMM_NVFP4 ? 16 : 8;
  const int sc_align = (sc_stride & 15) == 0 ? 16 : (sc_stride & 3) == 0 ? 4 : 1;
  const int cps = S::SEG / sc_want;  // chunks of a segment
  // stages of a chunk: whole ones, the k-blocks past K are zeros (of the codes, the scales and X)
  const int last_stages = (a.K - (nchunks - 1) * kExpChunk + 64 * SK - 1) / (64 * SK);
  const auto stages_of = [&](int c) { return c == nchunks - 1 ? last_stages : 4 / SK; };
  asm volatile("" ::"r"(nblocks), "r"(c0), "r"(c1), "r"(first), "r"(step), "r"(cps), "r"(last_stages));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 3) expert_tables(a, XT, bound, tstart, bad_flag);
  if (!a.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int items = *bad_flag ? 0 : tstart[a.E] * nblocks;

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
      const int box = min((it.rows + a.xunit - 1) / a.xunit, a.xmaps);
      for (int c = c0; c < c1 && ok; ++c) {
        const int nst = stages_of(c);
        for (int h = 0; h < nst; ++h, ++q) {
          if (q >= XS) ok = warp_wait(&mdone[s], par, ERR_TIMEOUT_PIPE, abort_flag);
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&xfull[s], uint32_t(SK * box * a.xunit) * 128u);
#pragma unroll
            for (int j = 0; j < SK; ++j)
              tma_load_2d(smem + S::OFF_X + s * S::SLOT_BYTES + j * XT * 128, &a.tmX[box - 1], &xfull[s],
                          c * kExpChunk + (h * SK + j) * 64, it.row);
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
    // stage of the codes; stage of dequantized weights; slot whose MMAs free it: that of stage q - AS
    // (counted from -AS: the slots of stages before the first are not waited for)
    int s = 0, as = 0, ms = (kb / SK - AS + XS) % XS;
    int sg = 0;                 // segments of scales so far
    uint32_t wpar = 0, mpar = kb / SK - AS < 0 ? 1 : 0;
    int q = kb / SK;            // this group's stage number; the first AS stages are free from the start
    bool ok = true;
    as = q % AS;
    for (int id = first; id < items && ok; id += step) {
      const Item it = item_of(id);
      // row of the weights (mod 2^32: only its bytes' place within a word is asked for)
      const uint32_t srow = uint32_t(it.e) * uint32_t(a.N) + uint32_t(min(it.n0 + trow, a.N - 1));
      const bool past = it.n0 + trow >= a.N;
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
              // a scale that is a normal fp16 (2^-14 .. 2^15) for the whole warp, or fp32 products; rows
              // past N count for none (their sums are not used)
              const uint32_t e8 = past ? 127u : (sc >> (8 * h)) & 255u;
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
        q += nst;  // this group's stage in the next chunk
        as = q % AS;
        ms += nst;
        if (ms >= XS) {
          ms -= XS;
          mpar ^= 1u;
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
    int i = 0;
    for (int id = first; id < items; id += step, ++i) {
      const Item it = item_of(id);
      const int b = i % NACC, u = i / NACC;
      const float gmul = FMT == GEMM_NVFP4 ? __ldg(a.gscale + it.e) : FMT == GEMM_INT4 ? 0.0625f : 1.0f;
      if (!warp_wait(&dfull[b], u & 1, ERR_TIMEOUT_MMA, abort_flag)) break;
      tc_fence_after();
      const int n = it.n0 + quarter * 32 + lane;  // this lane's weight row
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
        // a row of X at a time: 32 lanes' weight rows are 64 bytes of Y's row, whole sectors
        if (n < a.N) {
          uint16_t* y = a.Y + int64_t(it.row + x) * a.N + n;
          const int left = it.rows - x;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t y2 = pack_bf16x2(__uint_as_float(v[j]) * gmul, __uint_as_float(v[j + 1]) * gmul);
            if (j < left) y[0] = uint16_t(y2);
            if (j + 1 < left) y[a.N] = uint16_t(y2 >> 16);
            y += 2 * int64_t(a.N);
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
// dequantized in registers, and up to 8 rows of X as B, both in fp16.  Bound by HBM
// (0.53 to 0.63 bytes a weight) and by the instructions of the dequantization, which
// is why both operands are fp16: a pair of E2M1 codes is one conversion and one product
// there, against one conversion, two multiply-adds and a packing in bf16.  256 rows over 64
// experts of 1408 x 2048: INT4 (G = 64) 41 us, 2.4 TB/s; MXFP4 39.7 us; NVFP4 34.6 us (issue
// slots 50% busy, DRAM 28%: four warps a scheduler, dependent conversions and MMAs).
//
// A unit is 16 weight rows of one row tile; a step of it is 128 k.  A CTA takes a
// contiguous share of the units, each of its 16 warps a contiguous share of the CTA's
// steps: every SM streams the same number of bytes whatever N and K are.  Units that
// straddle warps are summed through shared memory, in warp order.
//
// X is staged once per row tile in the order of the MMA's B fragments, each row scaled
// by a power of two that puts its largest finite magnitude at 2^14: fp16 then holds
// bf16 exactly down to 2^-31 of that magnitude, and what is smaller to 2^-39 of it (INT4's
// elements that are staged / 16: 2^-27 and 2^-35).
// Two steps at a time: one alone left the warp waiting for its own results.  Codes come
// by cp.async, four to six steps ahead and on into the warp's next unit, into slots that
// the copying lane reads itself (no barrier, and a loop body of two steps: one unrolled
// over all that is in flight spent the short kernel's time on instruction fetches); scales
// two steps ahead into registers.
// Lane (g, c) (g = lane / 4, c = lane % 4) holds codes of rows g and g + 8; the k order
// inside an MMA is free, so its four k of each are four of the lane's own:
//   INT4   lane c takes G / 4 k of every group, so that an MMA stays inside a group: A is
//          1024 + q or 1024 + 16 q (one logic instruction a pair; X of the latter staged
//          / 16), and the group's fp32 sums lose what the 1024 and the zero point z added,
//          P + z Q from sums of the staged X, before the fp16 scale multiplies them.  The
//          sums round terms of up to 1264 |x| to fp32, about 2^-16 of the result where the
//          |q - z| are of middling size, more where an outlier of X meets q = z;
//   NVFP4  lane c takes 32 k in a row; A is the code times its block scale (exact);
//   MXFP4  the same, with the block scale relative to the largest of the row's step, and
//          the step's fp32 sums times that one; blocks under 2^-26 of it take another turn.
constexpr int kVecWarps = 16;
constexpr int kVecDepth = 6;
constexpr int kVecRows = 8;  // rows of X of a tile
constexpr int kVecRing = kVecWarps * kVecDepth * 1024;

// Shared memory: codes [warp][kVecDepth][2][32 lanes][16 bytes], sums of units that straddle
// warps, X fragments (all of K: MAX_STEPS is what this form serves).
template <int FMT>
struct VecShape {
  static constexpr int OFF_PART = kVecRing;
  static constexpr int OFF_X = OFF_PART + 2 * kVecWarps * 16 * kVecRows * 4;
  static constexpr int FRAG_BYTES = 2048;                                        // X fragments of a step
  static constexpr int STEP_BYTES = FRAG_BYTES + (FMT == GEMM_INT4 ? 256 : 0);  // and P, Q of its groups
  static constexpr int MAX_STEPS = (216 * 1024 - OFF_X) / STEP_BYTES;           // 52, INT4 46
};

__device__ __forceinline__ uint32_t ldg_u16(const void* p) { return __ldg(static_cast<const uint16_t*>(p)); }
__device__ __forceinline__ uint32_t ldg_u8(const void* p) { return __ldg(static_cast<const uint8_t*>(p)); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// FULL: K % 128 == 0, no step reaches past K (and a step's scales of a row are aligned words).
template <int FMT, int G, bool FULL>
__global__ void __launch_bounds__(kVecWarps * 32, 1) expert_gemv_kernel(const __grid_constant__ ExpertArgs a) {
  static_assert(FMT != GEMM_INT4 || G == 32 || G == 64 || G == 128, "group size");
  using V = VecShape<FMT>;
  constexpr int NG = FMT == GEMM_INT4 ? 128 / G : 1;    // groups of a step
  constexpr int WPG = 4 / NG;                           // words (8 k) of a lane per group
  extern __shared__ __align__(1024) uint8_t vec_smem[];
  __shared__ int bound[kMaxExperts + 4], tstart[kMaxExperts + 4];
  __shared__ int bad_flag;
  __shared__ uint32_t rtop[kVecRows];                     // largest finite magnitude of X's rows, fp32 bits
  // what undoes their scaling; MXFP4's sums are kept within fp32 by taking 2^-64 to 2^64 of it (rundo)
  // with each step's scales and only the rest (rscale) at the end
  __shared__ float rscale[kVecRows], rundo[kVecRows];
  __shared__ uint32_t rbad;                               // rows that hold a non-finite value, a bit each
  float (*part)[16][kVecRows] = reinterpret_cast<float (*)[16][kVecRows]>(vec_smem + V::OFF_PART);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int K = a.K, N = a.N;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.offsets) {
    if (warp == 0) expert_tables(a, kVecRows, bound, tstart, &bad_flag);
    __syncthreads();
    if (bad_flag) return;
  }
  const int tiles = a.offsets ? tstart[a.E] : (a.T + kVecRows - 1) / kVecRows;
  const int nrb = (N + 15) >> 4;                        // row blocks of an expert
  const int S = (K + 127) >> 7;                         // steps of a unit
  const int units = tiles * nrb, per = units / int(gridDim.x), more = units - per * int(gridDim.x);
  int u0 = int(blockIdx.x) * per + min(int(blockIdx.x), more);
  const int ulast = u0 + per + (int(blockIdx.x) < more);

  const int zw = (((FMT == GEMM_INT4 ? K / G : 8) + 7) >> 3) * 4;  // zero-point bytes of a row
  const int sw = FMT == GEMM_INT4 ? K / G * 2 : FMT == GEMM_NVFP4 ? K >> 4 : K >> 5;  // scale bytes of a row
  constexpr int SB = FMT == GEMM_INT4 ? 2 * NG : FMT == GEMM_NVFP4 ? 8 : 4;           // of a step
  const uint8_t* scales = FMT == GEMM_INT4 ? reinterpret_cast<const uint8_t*>(a.scales) : a.bscale;
  const uint32_t ring = smem_u32(vec_smem) + uint32_t(warp * kVecDepth * 1024 + lane * 16);
  const uint32_t xfrag = smem_u32(vec_smem) + uint32_t(V::OFF_X + lane * 16);
  int staged = -1;  // tile whose rows are in shared memory

  while (u0 < ulast) {
    // ---- a run of units of one row tile
    const int tile = u0 / nrb;
    const int u1 = min(ulast, (tile + 1) * nrb);
    int e = 0, row = tile * kVecRows, rows = min(kVecRows, a.T - row);
    if (a.offsets) {
      e = expert_of_tile(tstart, a.E, tile);
      const int r = bound[e + 1] - bound[e], nt = tstart[e + 1] - tstart[e];
      const int w = (r + nt - 1) / nt;  // the expert's rows, evenly over its tiles
      row = bound[e] + (tile - tstart[e]) * w;
      rows = min(w, bound[e + 1] - row);
    }
    const int nb0 = (u0 - tile * nrb) * 16, tot = (u1 - u0) * S;  // first weight row; steps of the CTA
    const auto first_of = [&](int w) { return int(int64_t(tot) * w / kVecWarps); };
    const float gmul = FMT == GEMM_NVFP4 ? __ldg(a.gscale + e) : 1.f;
    int at = first_of(warp);
    const int end = first_of(warp + 1);

    // ---- cursors over the run's steps, on into the next unit: codes and scales
    const auto row_of = [&](int u, int r) { return int64_t(e) * N + min(nb0 + u * 16 + r, N - 1); };
    const uint8_t *plo, *phi, *slo, *shi, *zlo, *zhi;
    int cu = 0, cj = 0, su = 0, sj = 0;  // unit and step of the next request and of the next scales
    uint32_t put = ring;
    const auto open_codes = [&]() {
      const int64_t rlo = row_of(cu, g), rhi = row_of(cu, g + 8);
      plo = a.packed + rlo * (K >> 1) + cj * 64 + (FMT == GEMM_INT4 ? c * (G / 8) : 16 * c);
      phi = plo + (rhi - rlo) * (K >> 1);
    };
    const auto open_scales = [&]() {
      const int64_t rlo = row_of(su, g), d = row_of(su, g + 8) - rlo;
      slo = scales + rlo * sw + sj * SB + (FMT == GEMM_NVFP4 ? 2 * c : FMT == GEMM_MXFP4 ? c : 0);
      shi = slo + d * sw;
      zlo = reinterpret_cast<const uint8_t*>(a.zeros) + rlo * zw;
      zhi = zlo + d * zw;
    };
    // a lane's 16 code bytes of each row, in word order; zeros past K
    const auto request = [&]() {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int k0 = cj * 128;
        const bool in = FULL || (FMT == GEMM_INT4 ? k0 + i * G < K : k0 + 32 * c < K);
        cp_async_zfill<16 / NG>(put + i * (16 / NG), in ? plo + i * (G / 2) : a.packed, in ? 16 / NG : 0);
        cp_async_zfill<16 / NG>(put + 512 + i * (16 / NG), in ? phi + i * (G / 2) : a.packed, in ? 16 / NG : 0);
      }
      plo += 64;
      phi += 64;
      put = put + 1024u == ring + kVecDepth * 1024u ? ring : put + 1024u;
      if (++cj == S) {
        cj = 0;
        ++cu;
        open_codes();
      }
    };
    // scales of rows g and g + 8 (fp16 per group, two E4M3 bytes, or an E8M0 byte) and the bytes
    // that hold the step's zero points (one for G >= 64, else two), as they are loaded: nothing
    // waits for them before the step that uses them
    struct Scales {
      uint32_t l[NG], h[NG], zl, zh;
    };
    const auto load_scales = [&](Scales& r) {
      if (FMT == GEMM_INT4 && FULL && NG > 1) {  // a row's scales of the step as words
#pragma unroll
        for (int i = 0; i < NG; i += 2) {
          r.l[i] = __ldg(reinterpret_cast<const uint32_t*>(slo + 2 * i));
          r.h[i] = __ldg(reinterpret_cast<const uint32_t*>(shi + 2 * i));
        }
      } else {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const bool in = FULL || (FMT == GEMM_INT4 ? (sj * NG + i) * 2 < sw : sj * 128 + 32 * c < K);
          r.l[i] = !in ? 0u : FMT == GEMM_MXFP4 ? ldg_u8(slo) : ldg_u16(slo + 2 * i);
          r.h[i] = !in ? 0u : FMT == GEMM_MXFP4 ? ldg_u8(shi) : ldg_u16(shi + 2 * i);
        }
      }
      slo += SB;
      shi += SB;
      r.zl = r.zh = 0x8888u;
      if (FMT == GEMM_INT4 && a.zeros) {
        const int b = (sj * NG) >> 1;
        r.zl = G == 32 ? ldg_u16(zlo + b) : ldg_u8(zlo + b);
        r.zh = G == 32 ? ldg_u16(zhi + b) : ldg_u8(zhi + b);
      }
      if (++sj == S) {
        sj = 0;
        ++su;
        open_scales();
      }
    };
    Scales r0 = {}, r1 = {};

    int u = 0, j = 0;  // unit and step in hand
    int todo = end;    // steps whose codes are still to be requested start here
    if (at < end) {    // the first codes are under way while X is staged
      u = at / S;
      j = at - u * S;
      cu = su = u;
      cj = sj = j;
      open_codes();
      open_scales();
      todo = min(end, at + kVecDepth);
#pragma unroll 1
      for (int i = 0; i < kVecDepth; ++i) {
        if (at + i < end) request();
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      load_scales(r0);
      if (at + 1 < end) load_scales(r1);
    }
    if (staged != tile) {
      // X, or X * act_inv_s, 256 k of a row at a time: the rows' largest finite magnitudes, then the fragments
      if (threadIdx.x < kVecRows) rtop[threadIdx.x] = 0;
      if (threadIdx.x == 0) rbad = 0;
      __syncthreads();  // also: the last run's readers are done
      const float* f = FMT == GEMM_MXFP4 ? a.inv_s : nullptr;
      // each row by two warps, alternate runs of 256 k
      constexpr int WPR = kVecWarps / kVecRows;
      const int m = warp / WPR, kend = m < rows ? S * 128 : 0;
      const uint16_t* xrow = a.X + int64_t(row + min(m, rows - 1)) * K;
      // four runs' loads in flight at once, twice over (the second time from L1)
      const auto pass = [&](auto&& use) {
#pragma unroll 1
        for (int kk = warp % WPR * 256 + lane * 8; kk - lane * 8 < kend; kk += 4 * WPR * 256) {
          uint4 r[4];
          float4 f0[4], f1[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int k = kk + q * WPR * 256;
            r[q] = k < K ? ldg_v4(xrow + k) : make_uint4(0, 0, 0, 0);
            if (FMT == GEMM_MXFP4) {
              f0[q] = f1[q] = make_float4(1.f, 1.f, 1.f, 1.f);
              if (f && k < K) {
                f0[q] = __ldg(reinterpret_cast<const float4*>(f + k));
                f1[q] = __ldg(reinterpret_cast<const float4*>(f + k) + 1);
              }
            }
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int k = kk + q * WPR * 256;
            const uint32_t w[4] = {r[q].x, r[q].y, r[q].z, r[q].w};
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[2 * i] = __uint_as_float(w[i] << 16);
              v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
            if (FMT == GEMM_MXFP4) {
              v[0] *= f0[q].x; v[1] *= f0[q].y; v[2] *= f0[q].z; v[3] *= f0[q].w;
              v[4] *= f1[q].x; v[5] *= f1[q].y; v[6] *= f1[q].z; v[7] *= f1[q].w;
            }
            use(k, v);
          }
        }
      };
      const auto largest = [&](uint32_t below) {  // of the magnitudes under `below`, fp32 bits
        uint32_t top = 0;
        pass([&](int, float (&v)[8]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
            top = max(top, b < below ? b : 0u);
          }
        });
        return __reduce_max_sync(0xffffffffu, top);
      };
      uint32_t top = largest(0x80000000u);
      if (top >= 0x7F800000u) {  // rare: a second look for the finite ones
        if (lane == 0) atomicOr(&rbad, 1u << m);
        top = largest(0x7F800000u);
      }
      if (lane == 0) atomicMax(&rtop[m], top);
      __syncthreads();
      const uint32_t fe = min(254u, 268u - max(rtop[m] >> 23, 1u));  // exponent field of 2^14 / 2^floor(log2 top)
      const float up = __uint_as_float(fe << 23);
      if (FMT == GEMM_MXFP4) {
        const uint32_t fu = min(191u, max(63u, fe));  // 127 -+ 64
        if (lane == 0) rundo[m] = __uint_as_float((254u - fu) << 23);
        if (lane == 0) rscale[m] = __uint_as_float((127u + fu - fe) << 23);
      } else if (lane == 0) {
        rscale[m] = __uint_as_float(fe == 254u ? 0x00400000u : (254u - fe) << 23);
      }
      pass([&](int k, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= up;
        const int p = (k & 127) >> 3;  // 8-k piece of the step: word w of lane cc
        uint8_t* step = vec_smem + V::OFF_X + (k >> 7) * V::STEP_BYTES;
        const bool in = k < S * 128;   // a run of 256 may pass an odd number of steps
        uint4 o;
        int w, cc;
        if constexpr (FMT == GEMM_INT4) {
          // {code i, code i + 4} of a word: x0 x4 | x1 x5 (of 16 q) | x2 x6 | x3 x7 (of 16 q)
          cc = (p * 8 % G) / (G / 4);
          w = (p * 8 / G) * WPG + (p * 8 % (G / 4)) / 8;
          o = make_uint4(pack_f16x2(v[0], v[4]), pack_f16x2(v[1] * 0.0625f, v[5] * 0.0625f), pack_f16x2(v[2], v[6]),
                         pack_f16x2(v[3] * 0.0625f, v[7] * 0.0625f));
          // what the group's sums hold of 1024, and the sum of X: both of the values as staged (those
          // that meet 16 q are X / 16), so that a rounding of X is not multiplied by 1024
          const auto pair = [](uint32_t h) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h));
            return t.x + t.y;
          };
          const float even = pair(o.x) + pair(o.z), odd = pair(o.y) + pair(o.w);
          float P = 1024.f * (even + odd), Q = even + 16.f * odd;
#pragma unroll
          for (int h = 1; h < G / 8; h <<= 1) {
            P += __shfl_xor_sync(0xffffffffu, P, h);
            Q += __shfl_xor_sync(0xffffffffu, Q, h);
          }
          if (in && p * 8 % G == 0)
            *reinterpret_cast<float2*>(step + V::FRAG_BYTES + ((p * 8 / G) * kVecRows + m) * 8) = make_float2(P, Q);
        } else {
          cc = p >> 2;
          w = p & 3;
          o = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
        }
        if (in) *reinterpret_cast<uint4*>(step + w * 512 + (4 * m + cc) * 16) = o;
      });
      staged = tile;
      __syncthreads();
    }

    // ---- the warp's steps
    // MXFP4: a step's sums, below 2^38, meet what undoes the scaling of columns 2 c and 2 c + 1 before
    // their scale of up to 2^127
    const float undo0 = FMT == GEMM_MXFP4 ? 0x1p-13f * rundo[2 * c] : 0.f;
    const float undo1 = FMT == GEMM_MXFP4 ? 0x1p-13f * rundo[2 * c + 1] : 0.f;
    // one step's products from its codes, scales and fragments
    const auto products = [&](int j, const uint4& cl4, const uint4& ch4, const Scales& r, float (&acc)[4]) {
      const uint32_t wl[4] = {cl4.x, cl4.y, cl4.z, cl4.w}, wh[4] = {ch4.x, ch4.y, ch4.z, ch4.w};
      const uint32_t xs = xfrag + uint32_t(j * V::STEP_BYTES);
      if (FMT == GEMM_INT4) {
        const uint32_t pq = smem_u32(vec_smem) + uint32_t(V::OFF_X + V::FRAG_BYTES + j * V::STEP_BYTES + c * 16);
        float d[4];  // the group's sums
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          constexpr uint32_t B = 0x64006400u;  // fp16 1024: a code under it is 1024 + q (or + 16 q)
          const uint32_t l8 = wl[w] >> 8, h8 = wh[w] >> 8;
          const uint32_t a0 = lop3_andor(wl[w], 0x000F000Fu, B), a2 = lop3_andor(wl[w], 0x00F000F0u, B);
          const uint32_t a1 = lop3_andor(wh[w], 0x000F000Fu, B), a3 = lop3_andor(wh[w], 0x00F000F0u, B);
          const uint32_t b0 = lop3_andor(l8, 0x000F000Fu, B), b2 = lop3_andor(l8, 0x00F000F0u, B);
          const uint32_t b1 = lop3_andor(h8, 0x000F000Fu, B), b3 = lop3_andor(h8, 0x00F000F0u, B);
          const uint4 x = ld_shared_v4(xs + uint32_t(w * 512));
          if (w % WPG == 0) d[0] = d[1] = d[2] = d[3] = 0.f;
          mma_f16_16816(d, a0, a1, a2, a3, x.x, x.y);
          mma_f16_16816(d, b0, b1, b2, b3, x.z, x.w);
          if (w % WPG == WPG - 1) {
            const int gi = w / WPG, nib = 4 * ((G == 128 ? (j & 1) : 0) + gi);
            const bool words = FULL && NG > 1;
            const uint32_t s2 = prmt_b32(r.l[words ? gi & ~1 : gi], r.h[words ? gi & ~1 : gi],
                                         words && (gi & 1) ? 0x7632 : 0x5410);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&s2));
            const float zl = __uint_as_float(lop3_andor(r.zl >> nib, 15u, 0x4B000000u)) - 8388608.f;
            const float zh = __uint_as_float(lop3_andor(r.zh >> nib, 15u, 0x4B000000u)) - 8388608.f;
            const uint4 t = ld_shared_v4(pq + uint32_t(gi * 64));  // P, Q of columns 2 c and 2 c + 1
            const float P0 = __uint_as_float(t.x), Q0 = __uint_as_float(t.y);
            const float P1 = __uint_as_float(t.z), Q1 = __uint_as_float(t.w);
            acc[0] = fmaf(f.x, fmaf(-zl, Q0, d[0] - P0), acc[0]);
            acc[1] = fmaf(f.x, fmaf(-zl, Q1, d[1] - P1), acc[1]);
            acc[2] = fmaf(f.y, fmaf(-zh, Q0, d[2] - P0), acc[2]);
            acc[3] = fmaf(f.y, fmaf(-zh, Q1, d[3] - P1), acc[3]);
          }
        }
      } else {
        // A = code times scale; fp16 pairs of the lane's two NVFP4 blocks, or of its MXFP4 block
        const auto mmas = [&](uint32_t l0, uint32_t l1, uint32_t h0, uint32_t h1, float (&d)[4]) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t sl = w < 2 ? l0 : l1, sh = w < 2 ? h0 : h1;
            const uint32_t a0 = h2_mul(e2m1x2_of_byte<0>(wl[w]), sl), a2 = h2_mul(e2m1x2_of_byte<1>(wl[w]), sl);
            const uint32_t b0 = h2_mul(e2m1x2_of_byte<2>(wl[w]), sl), b2 = h2_mul(e2m1x2_of_byte<3>(wl[w]), sl);
            const uint32_t a1 = h2_mul(e2m1x2_of_byte<0>(wh[w]), sh), a3 = h2_mul(e2m1x2_of_byte<1>(wh[w]), sh);
            const uint32_t b1 = h2_mul(e2m1x2_of_byte<2>(wh[w]), sh), b3 = h2_mul(e2m1x2_of_byte<3>(wh[w]), sh);
            const uint4 x = ld_shared_v4(xs + uint32_t(w * 512));
            mma_f16_16816(d, a0, a1, a2, a3, x.x, x.y);
            mma_f16_16816(d, b0, b1, b2, b3, x.z, x.w);
          }
        };
        if (FMT == GEMM_NVFP4) {
          const uint32_t fl = tc_e4m3x2(r.l[0] & 0x7F7Fu), fh = tc_e4m3x2(r.h[0] & 0x7F7Fu);
          mmas(prmt_b32(fl, fl, 0x1010), prmt_b32(fl, fl, 0x3232), prmt_b32(fh, fh, 0x1010),
               prmt_b32(fh, fh, 0x3232), acc);
        } else {
          // scale bytes + 1 of the blocks still to be taken, row g's in the low half; a block whose
          // codes are all zero counts for none (a NaN scale does)
          const bool zl = ((wl[0] | wl[1] | wl[2] | wl[3]) & 0x77777777u) == 0 && r.l[0] != 255u;
          const bool zh = ((wh[0] | wh[1] | wh[2] | wh[3]) & 0x77777777u) == 0 && r.h[0] != 255u;
          uint32_t rest = (zl ? 0u : r.l[0] + 1u) | (zh ? 0u : (r.h[0] + 1u) << 16);
          const auto turn = [&]() {
            // the rows' largest scales among them, and the blocks within 2^-26 of those
            uint32_t top = max_u16x2(rest, __shfl_xor_sync(0xffffffffu, rest, 1));
            top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t tl = top & 0xFFFFu, th = top >> 16, rl = rest & 0xFFFFu, rh = rest >> 16;
            const bool inl = rl != 0 && rl + 26u >= tl, inh = rh != 0 && rh + 26u >= th;
            // fp16 2^(13 + e - top): exponent field 28 + e - top
            const uint32_t fl = !inl ? 0u : rl == 256u ? 0x7E00u : (28u + rl - tl) << 10;
            const uint32_t fh = !inh ? 0u : rh == 256u ? 0x7E00u : (28u + rh - th) << 10;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mmas(fl * 0x10001u, fl * 0x10001u, fh * 0x10001u, fh * 0x10001u, d);
            // 2^(top - 127 - 13) in two factors: it may lie outside fp32's normal range
            const float ml = e8m0_f32(min(254u, max(tl, 1u) - 1u)), mh = e8m0_f32(min(254u, max(th, 1u) - 1u));
            acc[0] = fmaf(d[0] * undo0, ml, acc[0]);
            acc[1] = fmaf(d[1] * undo1, ml, acc[1]);
            acc[2] = fmaf(d[2] * undo0, mh, acc[2]);
            acc[3] = fmaf(d[3] * undo1, mh, acc[3]);
            rest = (inl ? 0u : rl) | ((inh ? 0u : rh) << 16);
          };
          turn();
#pragma unroll 1
          while (__any_sync(0xffffffffu, rest != 0)) turn();
        }
      }
    };
    const auto advance = [&](uint32_t p) { return p + 1024u == ring + kVecDepth * 1024u ? ring : p + 1024u; };
    uint32_t take = ring;
    bool begun = j == 0;  // the unit in hand, by this warp
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    while (at < end) {
      // one group a step was committed up to kVecDepth steps ahead: these two have landed
      asm volatile("cp.async.wait_group %0;" ::"n"(kVecDepth - 2) : "memory");
      const uint32_t take2 = advance(take);
      const uint4 l0 = ld_shared_v4(take), h0 = ld_shared_v4(take + 512);
      const Scales s0 = r0;
      if (j + 1 < S && at + 1 < end) {
        const uint4 l1 = ld_shared_v4(take2), h1 = ld_shared_v4(take2 + 512);
        const Scales s1 = r1;
        if (at + 2 < end) load_scales(r0);
        if (at + 3 < end) load_scales(r1);
        products(j, l0, h0, s0, acc);
        products(j + 1, l1, h1, s1, acc2);
        take = advance(take2);
        at += 2;
        j += 2;
        if (todo < end) { request(); ++todo; }
        asm volatile("cp.async.commit_group;" ::: "memory");
      } else {
        r0 = r1;
        if (at + 2 < end) load_scales(r1);
        products(j, l0, h0, s0, acc);
        take = take2;
        ++at;
        ++j;
      }
      if (todo < end) { request(); ++todo; }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (j < S && at < end) continue;
      // rows g and g + 8, columns 2 c and 2 c + 1: the CTA's result of the unit, or the warp's share
      const bool whole = begun && j == S;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int m = 2 * c + (q & 1), r = g + (q >> 1) * 8;
        float y = acc[q] + acc2[q];
        if (FMT != GEMM_NVFP4) {
          y *= rscale[m];
        } else {  // one large and the other small: their product first
          const bool apart = (gmul > 1.f) != (rscale[m] > 1.f);
          y = apart ? y * (gmul * rscale[m]) : y * gmul * rscale[m];
        }
        acc[q] = acc2[q] = 0.f;
        // slot 2 w: the unit was begun by an earlier warp; 2 w + 1: by this one
        if (!whole) {
          part[2 * warp + begun][r][m] = y;
        } else if (m < rows && nb0 + u * 16 + r < N) {
          a.Y[int64_t(row + m) * N + nb0 + u * 16 + r] = uint16_t(pack_bf16x2(y, y));
        }
      }
      ++u;
      j = 0;
      begun = true;
    }
    const uint32_t nonfinite = FMT == GEMM_NVFP4 ? 0u : rbad;  // this tile's: the next one is staged after the barrier
    __syncthreads();
    // ---- the warp that ends a unit begun by an earlier one adds the shares in warp order
    const int s0 = first_of(warp), us = s0 / S, ub = us * S;  // the unit of the warp's first step, and that unit's first
    if (s0 < end && s0 > ub && end >= ub + S) {
      float y[4] = {0.f, 0.f, 0.f, 0.f};  // outputs lane + 32 q of the unit's [16][8]
      int v = warp - 1;
      while (first_of(v) > ub) --v;
#pragma unroll 1
      for (; v <= warp; ++v) {
        const int b0 = first_of(v);
        if (b0 == first_of(v + 1)) continue;
        const float* share = &part[2 * v + (b0 <= ub)][0][0] + lane;
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] += share[32 * q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = (lane + 32 * q) >> 3, m = lane & 7;
        if (m < rows && nb0 + us * 16 + r < N) {
          a.Y[int64_t(row + m) * N + nb0 + us * 16 + r] = uint16_t(pack_bf16x2(y[q], y[q]));
        }
      }
    }
    if constexpr (FMT != GEMM_NVFP4) {
      if (nonfinite) {  // the same for every thread
        __syncthreads();  // after the stores above
        for (int i = threadIdx.x; i < (u1 - u0) * 16 * rows; i += kVecWarps * 32) {
          const int m = i % rows, n = nb0 + i / rows;
          if (!(nonfinite >> m & 1u) || n >= N) continue;
          const float y = nonfinite_terms<FMT>(a, row + m, int64_t(e) * N + n);
          a.Y[int64_t(row + m) * N + n] = uint16_t(pack_bf16x2(y, y));
        }
      }
    }
    u0 = u1;
  }
}

// ---------------------------------------------------------------------------
// Few rows, each by itself: multiply-adds on the CUDA cores, which take fewer
// instructions a weight here (1.5 to 2, and one more for a second row) than the MMA form
// above (about 2.5), need no staging and no barrier before the weights are under way.  One
// row of 11008 x 2048 MXFP4: 8.7 us, 1.4 TB/s (the launch and two dependent trips to memory
// are half of it: 2048 x 2048 takes 4.6 us); 8 rows over 64 experts of 1408 x 2048: MXFP4 9.5 us,
// INT4 9.3, NVFP4 8.2.
//
// A warp takes 8 weight rows over every `ksplit`-th 1024 k (lane: 32 consecutive k, 16
// bytes a row), all rows' codes by cp.async into slots that the lane reads itself, which
// leaves few enough registers for three CTAs on an SM; the grid's y is the row of X,
// whose expert every warp finds by itself from all the offsets.  A lane scales its own 32
// activations by a power of two that puts their largest finite magnitude at 2^14, so
// that fp16 holds them (exactly, down to 2^-31 of that magnitude), and undoes it in its
// fp32 sum.  INT4: 16 sum (1 + q / 16) x - (16 + z) sum x; E2M1: the converted code times
// x, the block scales on the sums.
constexpr int kRowWarps = 8;
constexpr int kRowRows = 8;

// v 2^e (e <= 252) in two factors: neither leaves fp32's range unless the result does.
__device__ __forceinline__ float times_pow2(float v, int e) {
  e = max(e, -252);
  const int h = e >> 1;
  return v * __uint_as_float(uint32_t(127 + h) << 23) * __uint_as_float(uint32_t(127 + e - h) << 23);
}

template <int FMT, int MT>
__global__ void __launch_bounds__(kRowWarps * 32, MT == 1 ? 3 : 2)
    expert_row_kernel(const __grid_constant__ ExpertArgs a, int ksplit) {
  __shared__ float part[kRowWarps][kRowRows * MT];
  // codes: [2][warp][row][32 lanes][16 bytes]; with 1/s, a run's 1024 of it: [warp][4096 bytes]
  extern __shared__ __align__(16) uint8_t row_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % ksplit, rb = blockIdx.x * (kRowWarps / ksplit) + warp / ksplit;
  const int n0 = rb * kRowRows, i0 = blockIdx.y;  // first weight row, first row of X
  const int K = a.K, N = a.N;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int e = 0;
  if (a.offsets) {
    int found = -1;
    bool bad = false;
    for (int b = lane; b < a.E; b += 32) {
      const int lo = __ldg(a.offsets + b), hi = __ldg(a.offsets + b + 1);
      bad |= lo < 0 || hi < lo || hi > a.T;
      if (lo <= i0 && i0 < hi) found = b;
    }
    if (__any_sync(0xffffffffu, bad)) {
      if (blockIdx.x == 0 && i0 == 0 && threadIdx.x == 0) report_error(ERR_OFFSETS);
      return;  // the same for every warp of the grid
    }
    e = __reduce_max_sync(0xffffffffu, found);
    if (e < 0) return;  // a row of no expert
  }
  const int64_t row0 = int64_t(e) * N + n0;
  const int rows = min(kRowRows, N - n0);  // none for the last CTA's spare warps
  bool bad = false;  // INT4: this lane has met a non-finite activation
  float acc[kRowRows][MT];
#pragma unroll
  for (int r = 0; r < kRowRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0.f;

  if (rows > 0) {
    const uint32_t slots = smem_u32(row_smem) + uint32_t(warp * kRowRows * 512 + lane * 16);
    const uint8_t* codes = a.packed + row0 * (K >> 1) + lane * 16;
    const int last = rows - 1;
    const auto request = [&](int k0, uint32_t dst) {  // a lane's 32 k are all in or all out: K % 32 == 0
      const bool in = k0 + lane * 32 < K;
      const uint8_t* p = codes + (k0 >> 1);
#pragma unroll
      for (int r = 0; r < kRowRows; ++r)
        cp_async_zfill<16>(dst + r * 512, in ? p + min(r, last) * int64_t(K >> 1) : a.packed, in ? 16 : 0);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // 1/s of a run, loaded along K: 32 lanes that each read 128 bytes in a row would touch 32
    // lines a load.  Piece c of lane l's eight lies at c ^ (l & 7), so that the reads spread over
    // the banks too.
    const uint32_t fslot = smem_u32(row_smem) + uint32_t(2 * kRowWarps * kRowRows * 512 + warp * 4096);
    const bool scaled = FMT == GEMM_MXFP4 && a.inv_s;
    const auto request_inv = [&](int k0) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int i = q * 32 + lane;  // piece of four
        const bool in = k0 + 4 * i < K;
        cp_async_zfill<16>(fslot + uint32_t((i & ~7) + ((i ^ (i >> 3)) & 7)) * 16, in ? a.inv_s + k0 + 4 * i : a.inv_s, in ? 16 : 0);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint32_t slot = slots;
    if (scaled) request_inv(sub * 1024);
    request(sub * 1024, slot);
#pragma unroll 1
    for (int k0 = sub * 1024; k0 < K; k0 += ksplit * 1024) {
      const uint32_t here = slot;
      slot = slot == slots ? slots + kRowWarps * kRowRows * 512 : slots;
      if (k0 + ksplit * 1024 < K) {
        request(k0 + ksplit * 1024, slot);
      } else {
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      if (scaled) {  // groups under way: 1/s and codes of the first run, or the other way round of a later one; the next codes
        if (k0 == sub * 1024)
          asm volatile("cp.async.wait_group 2;" ::: "memory");
        else
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
      }
      const int k = k0 + lane * 32;
      if (k >= K) break;  // only in a warp's last run
      // raw scales and zero-point words: nothing waits for them yet (nor for g, which, loaded
      // before the codes are under way, cost 8 rows over 64 experts 10.6 us instead of 8.2)
      const float g = FMT == GEMM_NVFP4 ? __ldg(a.gscale + e) : 1.f;
      uint32_t sc[kRowRows], zp[kRowRows];
      {
        const int ng = K >> a.log2g, gr = k >> a.log2g;
        const int sw = FMT == GEMM_INT4 ? 2 * ng : FMT == GEMM_NVFP4 ? K >> 4 : K >> 5;
        const uint8_t* sp = FMT == GEMM_INT4 ? reinterpret_cast<const uint8_t*>(a.scales) : a.bscale;
        sp += row0 * sw + (FMT == GEMM_INT4 ? 2 * gr : FMT == GEMM_NVFP4 ? k >> 4 : k >> 5);
        const uint32_t* zq = a.zeros + row0 * ((ng + 7) >> 3) + (gr >> 3);
#pragma unroll
        for (int r = 0; r < kRowRows; ++r) {
          const int64_t rr = min(r, last);
          sc[r] = FMT == GEMM_MXFP4 ? ldg_u8(sp + rr * sw) : ldg_u16(sp + rr * sw);
          zp[r] = FMT == GEMM_INT4 && a.zeros ? __ldg(zq + rr * ((ng + 7) >> 3)) : 0x88888888u;
        }
      }
      // the lane's activations (times 1/s) as fp16 pairs (INT4: {x0, x4} {x1, x5} {x2, x6} {x3, x7}
      // of eight), written over the bf16 ones
      uint32_t xh[MT][16];
      float back[MT], sum[MT];  // INT4: of the scaled activations
      int be[MT];               // back is 2^be
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 x = ldg_v4(a.X + int64_t(i0 + m) * K + k + 8 * q);
          xh[m][4 * q] = x.x; xh[m][4 * q + 1] = x.y; xh[m][4 * q + 2] = x.z; xh[m][4 * q + 3] = x.w;
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const auto quad = [&](int j) {  // elements 4 j to 4 j + 3
          const uint32_t u = xh[m][2 * j], v = xh[m][2 * j + 1];
          float4 f = make_float4(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u), __uint_as_float(v << 16),
                                 __uint_as_float(v & 0xFFFF0000u));
          if (scaled) {
            const uint4 i = ld_shared_v4(fslot + uint32_t(lane * 8 + (j ^ (lane & 7))) * 16);
            f.x *= __uint_as_float(i.x);
            f.y *= __uint_as_float(i.y);
            f.z *= __uint_as_float(i.z);
            f.w *= __uint_as_float(i.w);
          }
          return f;
        };
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 f = quad(j);
          const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
            top = max(top, b < 0x7F800000u ? b : 0u);
            if (FMT == GEMM_INT4) bad |= b >= 0x7F800000u;
          }
        }
        const uint32_t fe = min(254u, 268u - max(top >> 23, 1u));  // exponent field of 2^14 / 2^floor(log2 top)
        const float up = __uint_as_float(fe << 23);
        back[m] = __uint_as_float(fe == 254u ? 0x00400000u : (254u - fe) << 23);
        be[m] = 127 - int(fe);
        sum[m] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 f = quad(2 * q), h = quad(2 * q + 1);
          const float v[8] = {f.x * up, f.y * up, f.z * up, f.w * up, h.x * up, h.y * up, h.z * up, h.w * up};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (FMT == GEMM_INT4) {
              xh[m][4 * q + i] = pack_f16x2(v[i], v[i + 4]);
              sum[m] += v[i] + v[i + 4];
            } else {
              xh[m][4 * q + i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
            }
          }
        }
      }
      if (scaled) {
        if (k0 + ksplit * 1024 < K) {  // then no lane has left
          __syncwarp();                // every lane has taken this run's
          request_inv(k0 + ksplit * 1024);
        } else {
          asm volatile("cp.async.commit_group;" ::: "memory");
        }
        asm volatile("cp.async.wait_group 2;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      }
#pragma unroll
      for (int r = 0; r < kRowRows; ++r) {
        const uint4 w = ld_shared_v4(here + r * 512);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        float d[MT][2];  // E2M1: the lane's two blocks of 16; INT4: two chains
#pragma unroll
        for (int m = 0; m < MT; ++m) d[m][0] = d[m][1] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t p[4];
          if (FMT == GEMM_INT4) {
            constexpr uint32_t M = 0x03C003C0u, B = 0x3C003C00u;  // fp16 1 + q / 16: the code at bits 6-9
            p[0] = lop3_andor(ww[q] << 6, M, B);
            p[1] = lop3_andor(ww[q] << 2, M, B);
            p[2] = lop3_andor(ww[q] >> 2, M, B);
            p[3] = lop3_andor(ww[q] >> 6, M, B);
          } else {
            p[0] = e2m1x2_of_byte<0>(ww[q]);
            p[1] = e2m1x2_of_byte<1>(ww[q]);
            p[2] = e2m1x2_of_byte<2>(ww[q]);
            p[3] = e2m1x2_of_byte<3>(ww[q]);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float& s = d[m][q >> 1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              s = fma_f16_f32<0, 0>(p[j], xh[m][4 * q + j], s);
              s = fma_f16_f32<1, 1>(p[j], xh[m][4 * q + j], s);
            }
          }
        }
        // the scales meet the sums of the scaled activations first (below 2^50), what undoes that
        // scaling last: only the product itself may leave fp32's range
        float f0 = 0.f, f1 = 0.f, z = 0.f;
        if (FMT == GEMM_INT4) {
          f0 = __half2float(__ushort_as_half(uint16_t(sc[r])));
          z = 16.f + float((zp[r] >> (4 * ((k >> a.log2g) & 7))) & 15u);
        } else if (FMT == GEMM_NVFP4) {
          const uint32_t h = tc_e4m3x2(sc[r] & 0x7F7Fu);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          f0 = f.x;
          f1 = f.y;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (FMT == GEMM_INT4) {
            acc[r][m] += f0 * (16.f * (d[m][0] + d[m][1]) - z * sum[m]) * back[m];
          } else if (FMT == GEMM_NVFP4) {
            // one of g and back large and the other small: their product first
            const float t = f0 * d[m][0] + f1 * d[m][1];
            const bool apart = (g > 1.f) != (back[m] > 1.f);
            acc[r][m] += t * (apart ? g * back[m] : g) * (apart ? 1.f : back[m]);
          } else {
            const float t = times_pow2(d[m][0] + d[m][1], int(sc[r]) - 127 + be[m]);
            acc[r][m] += sc[r] == 255u ? __uint_as_float(0x7FC00000u) : t;
          }
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // ---- sums over the lanes: eight rows at once, half of them handed over at each of three exchanges
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = acc[r][m];
#pragma unroll
    for (int h = 4; h >= 1; h >>= 1) {
      const bool up = (lane & (h * 4)) != 0;
#pragma unroll
      for (int r = 0; r < h; ++r) {
        const float give = up ? v[r] : v[r + h], keep = up ? v[r + h] : v[r];
        v[r] = keep + __shfl_xor_sync(0xffffffffu, give, h * 4);
      }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    if ((lane & 3) == 0) part[warp][(lane >> 2) * MT + m] = v[0];  // row lane / 4
  }
  // a row of X with non-finite values: some lane of the row block's warps has met them
  const bool nonfinite = __syncthreads_or(bad);
  const int t = threadIdx.x;
  if (t < kRowWarps / ksplit * kRowRows * MT) {
    const int b = t / (kRowRows * MT), r = t / MT % kRowRows, m = t % MT;
    const int n = (blockIdx.x * (kRowWarps / ksplit) + b) * kRowRows + r;
    float y = 0.f;
    for (int w = 0; w < ksplit; ++w) y += part[b * ksplit + w][r * MT + m];
    if constexpr (FMT == GEMM_INT4) {
      if (nonfinite && n < N) {
        const float inf = nonfinite_terms<FMT>(a, i0 + m, int64_t(e) * N + n);
        if (!isfinite(inf)) y = inf;
      }
    }
    if (n < N) a.Y[int64_t(i0 + m) * N + n] = uint16_t(pack_bf16x2(y, y));
  }
}

}  // namespace wq

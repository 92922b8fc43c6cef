// gemm_mxf4.cuh -- MXFP4 W4A4 GEMM on the block-scaled FP4 tensor cores
// (tcgen05.mma kind::mxf4, one E8M0 scale per 32 elements of each operand):
//   Y[m, n] = sum_b 2^(ex[m,b] + ew[n,b]) sum_{k in b} e2m1(xq[m,k]) e2m1(wq[n,k])
// X was packed to MXFP4 along K just before (mxfp4_pack_kernel).
//
// Persistent, one CTA per SM over 128 x 192 tiles of Y; k-blocks of 256 elements
// (128 bytes a row, one swizzle atom).  192 columns because two accumulators and the
// scales fit the 512 columns of tensor memory, and because a k-block's codes then take 52
// bytes a clock into the SM at the full FP4 rate (128 x 128 tiles need 64, what an SM takes).
//   warp 0      TMA: codes of X [128 x 128 B] and W [192 x 128 B]
//   warp 1      TMEM allocation and the MMA issuer (4 MMAs of K = 64 per k-block)
//   warps 4-7   scales: global -> registers (two k-blocks ahead) -> tensor memory, one
//               lane quarter each (every quarter holds all rows' scales)
//   warps 8-11  epilogue of one accumulator while the other is filled
// A word of scales (4 bytes, K = 128) of row r lies at column r / 32 of its block and
// lane r % 32 of every quarter; the instruction descriptor names the half of it (two
// bytes, K = 64) that an MMA takes.
// Bound by the way of the scales: each of the four warps reads all 320 rows' of a k-block, 8
// bytes a row at a stride of K / 32.  2048 x 11008 x 2048 takes 52 us with the pack of X (1780
// TFLOP/s; 14.8 us at the FP4 rate of a library product, 6.2 PFLOP/s); with constants in place of
// the scales read 33.5 us, without the stores of Y 50.4.  Few rows: 10.9 us for 1 x 11008 x 2048,
// 11.7 for 128, 18.6 for 512.
#pragma once

#include "experts.cuh"
#include "gemm_fp4.cuh"

namespace wq {

struct Mxf4Shape {
  static constexpr int BN = 192, STAGES = 5;
  static constexpr int A_BYTES = kGemmBM * kFp4BK / 2;  // 16 KB
  static constexpr int B_BYTES = BN * kFp4BK / 2;       // 24 KB
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int THREADS = 384;
  static constexpr int SF_STAGES = 4;
  static constexpr int AR = kGemmBM / 32, BR = BN / 32;  // columns of one word of all rows
  static constexpr int SF_COLS = 2 * (AR + BR);          // two words a row and k-block
  static constexpr int ACC_COLS = 2 * BN;
  static constexpr int TMEM_COLS = 512;
  static_assert(ACC_COLS + SF_STAGES * SF_COLS <= TMEM_COLS, "tensor memory budget");
  static constexpr int YBOX_BYTES = 32 * 32 * 2;
  static constexpr int Y_BYTES = 4 * 2 * YBOX_BYTES;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + Y_BYTES + 512 + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
};

struct Mxf4Args {
  CUtensorMap tmA;     // X codes u8 [M, K/2], box {128 B, 128}, 128B swizzle
  CUtensorMap tmB;     // W codes u8 [N, K/2], box {128 B, 192}, 128B swizzle
  CUtensorMap tmY;     // Y bf16 [M, N], box {32, 32}, 64B swizzle (used iff y_tma)
  const uint8_t* sfa;  // X e8m0 [M, K/32]
  const uint8_t* sfb;  // W e8m0 [N, K/32]
  uint16_t* Y;         // bf16 [M, N]
  int y_tma;           // N % 8 == 0 and Y 16-byte aligned
  int M, N, K;         // K % 64 == 0
};

// Instruction descriptor: E2M1 x E2M1 with E8M0 block scales (bytes sf, sf + 1 of a word), fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int sf) {
  return (uint32_t(sf) << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (1u << 23) | (uint32_t(M >> 4) << 24) |
         (uint32_t(sf) << 29);
}

__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p; }" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__global__ void __launch_bounds__(Mxf4Shape::THREADS, 1) gemm_mxf4_kernel(const __grid_constant__ Mxf4Args a) {
  using S = Mxf4Shape;
  constexpr int STAGES = S::STAGES, BN = S::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  uint8_t* ybox = smem + STAGES * S::STAGE_BYTES;  // epilogue boxes of Y (1024-byte aligned)
  uint64_t* bars = reinterpret_cast<uint64_t*>(ybox + S::Y_BYTES);
  uint64_t* full = bars;                          // codes landed
  uint64_t* empty = full + STAGES;                // MMAs of the stage finished
  uint64_t* sfready = empty + STAGES;             // scales in tensor memory
  uint64_t* sfempty = sfready + S::SF_STAGES;     // MMAs that read them finished
  uint64_t* acc_full = sfempty + S::SF_STAGES;    // [2] accumulator complete
  uint64_t* acc_empty = acc_full + 2;             // [2] accumulator drained
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int nkb = (a.K + kFp4BK - 1) / kFp4BK;
  const int n_tiles = (a.N + BN - 1) / BN, m_tiles = (a.M + kGemmBM - 1) / kGemmBM;
  const int tiles = n_tiles * m_tiles;
  if (warp == 0) {
    if (lane < STAGES) { mbar_init(&full[lane], 1); mbar_init(&empty[lane], 1); }
    if (lane < S::SF_STAGES) { mbar_init(&sfready[lane], 4); mbar_init(&sfempty[lane], 1); }
    if (lane < 2) { mbar_init(&acc_full[lane], 1); mbar_init(&acc_empty[lane], 4); }
    fence_mbar_init();
    if (lane == 0) {
      *abort_flag = 0;
      prefetch_tmap(&a.tmA);
      prefetch_tmap(&a.tmB);
      if (a.y_tma) prefetch_tmap(&a.tmY);
    }
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, S::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == 0) {
    // ---------------------------------------------------------- codes
    int q = 0, s = 0;
    uint32_t par = 1;  // parity of the stage's last use (the first use waits for none)
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const int m0 = (t / n_tiles) * kGemmBM, n0 = (t % n_tiles) * BN;
      for (int kb = 0; kb < nkb; ++kb, ++q) {
        if (q >= STAGES) ok = warp_wait(&empty[s], par, ERR_TIMEOUT_PIPE, abort_flag);
        if (!ok) break;
        if (elect_one()) {
          uint8_t* st = smem + s * S::STAGE_BYTES;
          mbar_arrive_expect_tx(&full[s], S::STAGE_BYTES);
          tma_load_2d(st, &a.tmA, &full[s], kb * (kFp4BK / 2), m0);
          tma_load_2d(st + S::A_BYTES, &a.tmB, &full[s], kb * (kFp4BK / 2), n0);
        }
        __syncwarp();
        if (++s == STAGES) {
          s = 0;
          par ^= 1u;
        }
      }
    }
    if (!ok) {  // let copies already issued land before the CTA leaves
      for (int k = (q > STAGES ? q - STAGES : 0); k < q; ++k)
        mbar_wait(&full[k % STAGES], (k / STAGES) & 1, ERR_TIMEOUT_TMA, nullptr);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const uint64_t ad0 = desc_kmajor_sw128(sbase), bd0 = desc_kmajor_sw128(sbase + uint32_t(S::A_BYTES));
    int q = 0, i = 0, s = 0;
    uint32_t par = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++i) {
      const int b = i & 1, u = i >> 1;
      if (u > 0) ok = warp_wait(&acc_empty[b], (u - 1) & 1, ERR_TIMEOUT_PIPE, abort_flag);
      if (!ok) break;
      const uint32_t dacc = tmem + uint32_t(b * BN);
      for (int kb = 0; kb < nkb; ++kb, ++q) {
        const int f = q % S::SF_STAGES;
        const uint32_t fpar = (q / S::SF_STAGES) & 1;
        const bool r1 = mbar_try_wait(&full[s], par), r2 = mbar_try_wait(&sfready[f], fpar);
        if (!__all_sync(0xffffffffu, r1 && r2))
          ok = warp_wait(&full[s], par, ERR_TIMEOUT_TMA, abort_flag) &&
               warp_wait(&sfready[f], fpar, ERR_TIMEOUT_PIPE, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = ad0 + uint64_t(uint32_t(s * (S::STAGE_BYTES >> 4)));
          const uint64_t bd = bd0 + uint64_t(uint32_t(s * (S::STAGE_BYTES >> 4)));
          const uint32_t sfa = tmem + uint32_t(S::ACC_COLS + f * S::SF_COLS), sfb = sfa + 2 * S::AR;
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4)  // K = 64: 32 bytes inside the swizzle atom, half a word of scales
            umma_mxf4(dacc, ad + uint64_t(2 * k4), bd + uint64_t(2 * k4), idesc_mxf4(kGemmBM, BN, 2 * (k4 & 1)),
                      sfa + (k4 >> 1) * S::AR, sfb + (k4 >> 1) * S::BR, uint32_t(kb | k4));
          umma_commit(&empty[s]);
          umma_commit(&sfempty[f]);
        }
        __syncwarp();
        if (++s == STAGES) {
          s = 0;
          par ^= 1u;
        }
      }
      if (elect_one()) umma_commit(&acc_full[b]);  // also after an abort: completes when the issued MMAs are done
      __syncwarp();
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------- scales
    const int quarter = warp & 3;
    const int stride = a.K >> 5;                  // scale bytes of a row
    const bool wide = (a.K & 255) == 0;           // a k-block's eight bytes are aligned
    const uint32_t dst0 = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(S::ACC_COLS);
    // the k-block's scales of row `row` of `rows` (zeros past the rows and past K)
    const auto fetch = [&](const uint8_t* sf, int row, int rows, int kb) {
      uint2 v = make_uint2(0, 0);
      if (row >= rows) return v;
      const uint8_t* p = sf + int64_t(row) * stride + kb * 8;
      if (wide) return __ldg(reinterpret_cast<const uint2*>(p));
      const int n = min(8, stride - kb * 8);      // even: K % 64 == 0
      if (n > 0) v.x = __ldg(reinterpret_cast<const uint16_t*>(p));
      if (n > 2) v.x |= uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p + 2))) << 16;
      if (n > 4) v.y = __ldg(reinterpret_cast<const uint16_t*>(p + 4));
      if (n > 6) v.y |= uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p + 6))) << 16;
      return v;
    };
    // the k-blocks of this CTA's tiles in order; `t`, `kb` name the next one to fetch
    int t = blockIdx.x, kb = 0;
    const auto next = [&](uint2 (&v)[S::AR + S::BR]) {
      if (t >= tiles) return;
      const int m0 = (t / n_tiles) * kGemmBM, n0 = (t % n_tiles) * BN;
#pragma unroll
      for (int c = 0; c < S::AR; ++c) v[c] = fetch(a.sfa, m0 + 32 * c + lane, a.M, kb);
#pragma unroll
      for (int c = 0; c < S::BR; ++c) v[S::AR + c] = fetch(a.sfb, n0 + 32 * c + lane, a.N, kb);
      if (++kb == nkb) {
        kb = 0;
        t += gridDim.x;
      }
    };
    const int64_t total = blockIdx.x < tiles ? int64_t((tiles - 1 - blockIdx.x) / gridDim.x + 1) * nkb : 0;
    uint2 v[2][S::AR + S::BR];
    next(v[0]);
    next(v[1]);
    bool ok = true;
    for (int64_t q0 = 0; q0 < total && ok; q0 += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t q = q0 + h;
        if (q >= total) break;
        const int f = int(q % S::SF_STAGES);
        if (q >= S::SF_STAGES)
          ok = warp_wait(&sfempty[f], uint32_t(q / S::SF_STAGES - 1) & 1u, ERR_TIMEOUT_PIPE, abort_flag);
        if (!ok) break;
        tc_fence_after();
        uint32_t w[S::SF_COLS];
#pragma unroll
        for (int c = 0; c < S::AR; ++c) { w[c] = v[h][c].x; w[S::AR + c] = v[h][c].y; }
#pragma unroll
        for (int c = 0; c < S::BR; ++c) {
          w[2 * S::AR + c] = v[h][S::AR + c].x;
          w[2 * S::AR + S::BR + c] = v[h][S::AR + c].y;
        }
        static_assert(S::SF_COLS == 20, "stores of 8, 8 and 4 columns");
        const uint32_t dst = dst0 + uint32_t(f * S::SF_COLS);
        tmem_st8(dst, w);
        tmem_st8(dst + 8, w + 8);
        tmem_st4(dst + 16, w + 16);
        next(v[h]);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfready[f]);
      }
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------- epilogue
    const int quarter = warp & 3;
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    int i = 0, nbox = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
      const int b = i & 1, u = i >> 1;
      if (!warp_wait(&acc_full[b], u & 1, ERR_TIMEOUT_MMA, abort_flag)) break;
      tc_fence_after();
      const int m0 = (t / n_tiles) * kGemmBM, n0 = (t % n_tiles) * BN;
      const int row = m0 + quarter * 32 + lane;
      for (int c = 0; c < BN && n0 + c < a.N; c += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + lane_base + uint32_t(b * BN + c), v);
        if (a.y_tma) {
          // the warp's 32 x 32 box (row = lane) through shared memory and one TMA store; box
          // buffers alternate, the one used two boxes ago must have been read
          uint8_t* box = ybox + (quarter * 2 + (nbox & 1)) * S::YBOX_BYTES;
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          const uint32_t rbase = smem_u32(box) + uint32_t(lane * 64);
#pragma unroll
          for (int p = 0; p < 4; ++p) {  // 16-byte piece p of the row, at its 64B-swizzled place
            uint4 o;
            o.x = pack_bf16x2(__uint_as_float(v[8 * p + 0]), __uint_as_float(v[8 * p + 1]));
            o.y = pack_bf16x2(__uint_as_float(v[8 * p + 2]), __uint_as_float(v[8 * p + 3]));
            o.z = pack_bf16x2(__uint_as_float(v[8 * p + 4]), __uint_as_float(v[8 * p + 5]));
            o.w = pack_bf16x2(__uint_as_float(v[8 * p + 6]), __uint_as_float(v[8 * p + 7]));
            st_shared_v4(rbase + uint32_t((p ^ ((lane >> 1) & 3)) << 4), o);
          }
          fence_proxy_async_smem();  // generic-proxy stores -> visible to the TMA
          __syncwarp();
          if (lane == 0 && m0 + quarter * 32 < a.M) {  // rows and columns past M and N are clipped by the TMA
            tma_store_2d(&a.tmY, box, n0 + c, m0 + quarter * 32);
            bulk_commit();
          }
          ++nbox;
        } else if (row < a.M) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (n0 + c + j < a.N)
              a.Y[int64_t(row) * a.N + n0 + c + j] = uint16_t(pack_bf16x2(__uint_as_float(v[j]), __uint_as_float(v[j])));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
    }
    if (lane == 0) bulk_wait_all();  // the Y stores are complete before the CTA leaves
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, S::TMEM_COLS);
  }
}

}  // namespace wq

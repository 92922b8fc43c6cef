// experts.cuh -- products grouped by expert over a stack of 4-bit packs:
// Y[i] = X[i] W_e^T for offsets[e] <= i < offsets[e + 1].
#pragma once

#include <cuda_fp16.h>

#include "gemm_tcgen05.cuh"
#include "mxfp4.cuh"
#include "wq_common.cuh"

namespace wq {

struct ExpertArgs {
  const uint16_t* X;       // bf16 [T, K]
  const int* offsets;      // [E + 1], or null: one expert over all T rows
  const float* inv_s;      // fp32 [K] or null: multiplies column k of X
  const uint8_t* packed;   // K / 2 bytes per row, rows [E * N]
  const uint16_t* scales;  // INT4 fp16 [E * N, K / G]
  const uint32_t* zeros;   // INT4 [E * N, ceil(K / G / 8)] or null (symmetric, z = 8)
  const uint8_t* bscale;   // NVFP4 E4M3 [E * N, K / 16]; MXFP4 E8M0 [E * N, K / 32]
  const float* gscale;     // NVFP4 fp32 [E]
  uint16_t* Y;             // bf16 [T, N]
  int E, N, K, T;
  int log2g;
};

// Simple form: one warp per (row i, weight row n).
template <int FMT>
__global__ void __launch_bounds__(256) experts_simple_kernel(const ExpertArgs a) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.y;
  bool bad = false;
  for (int e = threadIdx.x; a.offsets && e < a.E; e += blockDim.x)
    bad |= a.offsets[e] < 0 || a.offsets[e] > a.offsets[e + 1] || a.offsets[e + 1] > a.T;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) report_error(ERR_OFFSETS);
    return;
  }
  int lo = 0, hi = a.E;  // the last e with offsets[e] <= i
  if (a.offsets) {
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.offsets[mid] <= i) lo = mid; else hi = mid;
    }
    if (i < a.offsets[0] || i >= a.offsets[lo + 1]) return;
  }
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const int64_t row = int64_t(lo) * a.N + n;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(a.packed + row * (a.K / 2));
  float acc = 0.f;
  for (int j = lane; j < a.K / 8; j += 32) {
    const uint32_t w = words[j];
    float sc, z = 0.f;
    if (FMT == GEMM_INT4) {
      const int ng = a.K >> a.log2g, g = (8 * j) >> a.log2g;
      sc = __half2float(__ushort_as_half(a.scales[row * ng + g]));
      z = a.zeros ? float((a.zeros[row * ((ng + 7) >> 3) + (g >> 3)] >> (4 * (g & 7))) & 15u) : 8.f;
    } else if (FMT == GEMM_NVFP4) {
      sc = e4m3_decode_pos(a.bscale[row * (a.K / 16) + j / 2] & 0x7F);
    } else {
      sc = e8m0_f32(a.bscale[row * (a.K / 32) + j / 4]);
    }
    const uint4 xv = ldg_v4(a.X + int64_t(i) * a.K + 8 * j);
    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
    const uint4 dv = dequant_word_nvfp4(w, 0x3F803F80u);
    const uint32_t dw[4] = {dv.x, dv.y, dv.z, dv.w};
    float part = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float x = q & 1 ? __uint_as_float(xw[q / 2] & 0xFFFF0000u) : __uint_as_float(xw[q / 2] << 16);
      if (a.inv_s) x *= __ldg(a.inv_s + 8 * j + q);
      const float v = FMT == GEMM_INT4 ? float((w >> (4 * q)) & 15u) - z
                                       : (q & 1 ? __uint_as_float(dw[q / 2] & 0xFFFF0000u) : __uint_as_float(dw[q / 2] << 16));
      part = fmaf(x, v, part);
    }
    acc = fmaf(part, sc, acc);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if (FMT == GEMM_NVFP4) acc *= a.gscale[lo];
  if (lane == 0) a.Y[int64_t(i) * a.N + n] = uint16_t(pack_bf16x2(acc, acc));
}

}  // namespace wq

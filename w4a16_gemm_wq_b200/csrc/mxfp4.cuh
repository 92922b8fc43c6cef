// mxfp4.cuh -- MXFP4 (OCP microscaling) pack and its reading back.
//
// Per block of 32 consecutive k with m = max|w'| (w' = W, or W s in fp32):
//   e = clamp(floor(log2 m) - 2, -127, 127)   (2 = exponent of E2M1's largest value, 6)
//   code = nearest E2M1 of w' / 2^e, ties to the even code, saturating at 6, sign kept
//   scale byte = e + 127 (E8M0);  an all-zero block gets e = -127;
//   a block that holds an infinity or a NaN gets the byte 255 (E8M0 NaN) and zero codes.
// floor(log2 m) is m's exponent field, and the division by 2^e is exact (an
// exact multiplication by 2^-e: w' / 2^e is below 8 and only loses bits below
// fp32's smallest subnormal, far under E2M1's first tie at 0.25), so the pack
// takes integer and exact decisions only.
//
// Both directions are streaming passes bound by HBM (2.53 bytes a weight).  One
// thread takes 8 weights (a 16-byte load or store and one word of codes), four
// neighbouring lanes a block, so all accesses of a warp are contiguous; kMxUnroll
// loads per thread are in flight at once.  16384 x 8192: pack 60 us, values 62 us, 5.6 TB/s
// each way (85% of the measured copy; the pack's integer pipe is 75% busy).
#pragma once

#include "gemm_tcgen05.cuh"
#include "quant.cuh"
#include "wq_common.cuh"

namespace wq {

constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 4;

// bf16x2 {2^e, 2^e} of an E8M0 byte: e = byte - 127; byte 0 is the bf16 subnormal 2^-127, 255 NaN.
__device__ __forceinline__ uint32_t e8m0_bf16x2(uint32_t b) {
  const uint32_t h = b == 0 ? 0x0040u : b == 255 ? 0x7FC0u : b << 7;
  return h | (h << 16);
}
__device__ __forceinline__ float e8m0_f32(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}

__global__ void __launch_bounds__(kMxThreads) mxfp4_pack_kernel(const uint16_t* __restrict__ A,
                                                                const float* __restrict__ s, uint64_t words,
                                                                uint32_t row_words, uint32_t* __restrict__ codes,
                                                                uint8_t* __restrict__ bscale) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint64_t stride = uint64_t(gridDim.x) * kMxThreads;
  // every lane of a warp runs the same number of rounds: the blocks' maxima are shuffles
  for (uint64_t base = uint64_t(blockIdx.x) * kMxThreads; base < words; base += kMxUnroll * stride) {
    uint4 raw[kMxUnroll];
#pragma unroll
    for (int q = 0; q < kMxUnroll; ++q) {
      const uint64_t u = base + threadIdx.x + q * stride;
      raw[q] = u < words ? ldg_stream_v4(A + u * 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < kMxUnroll; ++q) {
      const uint64_t u = base + threadIdx.x + q * stride;
      const uint32_t r[4] = {raw[q].x, raw[q].y, raw[q].z, raw[q].w};
      float w[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[2 * j] = __uint_as_float(r[j] << 16);
        w[2 * j + 1] = __uint_as_float(r[j] & 0xFFFF0000u);
      }
      uint32_t top;  // bit pattern of the lane's largest magnitude (fp32; patterns order like magnitudes, NaN highest)
      if (s) {
        const uint64_t uc = u < words ? u : 0;
        const uint32_t c = words <= 0xFFFFFFFFull ? uint32_t(uc) % row_words : uint32_t(uc % row_words);
        const float4 s0 = __ldg(reinterpret_cast<const float4*>(s + uint64_t(c) * 8));
        const float4 s1 = __ldg(reinterpret_cast<const float4*>(s + uint64_t(c) * 8) + 1);
        const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
        top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[j] = __fmul_rn(w[j], sv[j]);
          top = max(top, __float_as_uint(w[j]) & 0x7FFFFFFFu);
        }
      } else {
        const uint32_t a = max_u16x2(r[0] & 0x7FFF7FFFu, r[1] & 0x7FFF7FFFu);
        const uint32_t b = max_u16x2(r[2] & 0x7FFF7FFFu, r[3] & 0x7FFF7FFFu);
        const uint32_t c = max_u16x2(a, b);
        top = max(c & 0xFFFFu, c >> 16) << 16;
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t field = top >> 23;  // biased exponent of the block's maximum
      const bool bad = field == 255;
      const uint32_t byte = bad ? 255u : field > 2 ? field - 2 : 0u;
      const float inv = __uint_as_float(bad ? 0u : (254u - byte) << 23);  // 2^-e
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) word |= e2m1x2_rn_sat(__fmul_rn(w[2 * j], inv), __fmul_rn(w[2 * j + 1], inv)) << (8 * j);
      if (bad) word = 0;
      if (u < words) {
        codes[u] = word;
        if ((threadIdx.x & 3) == 0) bscale[u >> 2] = uint8_t(byte);
      }
    }
  }
}

// X 1/s in bf16, for the W4A16 product: one rounding of 2^-8 at most a term, as the product would
// otherwise round the weight times 1/s, but once an element of X instead of once for every
// weight in every row tile (bf16 because the MMA takes both operands in one type, and fp16 has
// no room for the weights' scales; a second bf16 term for the rest would double the products).
__global__ void __launch_bounds__(kMxThreads) mxfp4_scale_kernel(const uint16_t* __restrict__ X,
                                                                 const float* __restrict__ s, uint64_t words,
                                                                 uint32_t row_words, uint16_t* __restrict__ out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (uint64_t u = uint64_t(blockIdx.x) * kMxThreads + threadIdx.x; u < words; u += uint64_t(gridDim.x) * kMxThreads) {
    const uint4 raw = ldg_v4(X + u * 8);
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
    const float4* f = reinterpret_cast<const float4*>(s) + 2 * (u % row_words);
    const float4 f0 = __ldg(f), f1 = __ldg(f + 1);
    const float fv[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = pack_bf16x2(__uint_as_float(r[j] << 16) * fv[2 * j], __uint_as_float(r[j] & 0xFFFF0000u) * fv[2 * j + 1]);
    reinterpret_cast<uint4*>(out)[u] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// The values of a pack in bf16: exact (at most two significant bits, exponents -128 .. 129; under
// scale bytes of 253 and 254, which the pack never writes, codes of 2^128 and more are infinities).
__global__ void __launch_bounds__(kMxThreads) mxfp4_unpack_kernel(const uint32_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ bscale, uint64_t words,
                                                                  uint16_t* __restrict__ out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint64_t stride = uint64_t(gridDim.x) * kMxThreads;
  for (uint64_t base = uint64_t(blockIdx.x) * kMxThreads + threadIdx.x; base < words; base += kMxUnroll * stride) {
    uint32_t w[kMxUnroll], b[kMxUnroll];
#pragma unroll
    for (int q = 0; q < kMxUnroll; ++q) {
      const uint64_t u = base + q * stride;
      w[q] = u < words ? __ldg(codes + u) : 0u;
      b[q] = u < words ? __ldg(bscale + (u >> 2)) : 0u;
    }
#pragma unroll
    for (int q = 0; q < kMxUnroll; ++q) {
      const uint64_t u = base + q * stride;
      if (u < words) reinterpret_cast<uint4*>(out)[u] = dequant_word_nvfp4(w[q], e8m0_bf16x2(b[q]));
    }
  }
}

}  // namespace wq

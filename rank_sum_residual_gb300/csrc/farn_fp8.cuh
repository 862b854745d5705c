// E4M3 codes with an fp32 scale per block: the arithmetic that the block
// quantisation and the 8-bit cache share.
#pragma once

#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "farn_kernels.cuh"

namespace farn {

constexpr int kFp8Block = 128;    // elements of a row under one scale

// scale = amax / 448 and inv = 448 / amax, both 1 for an all-zero block.  inv
// stays finite for an amax below 2^-119, so that zeros next to it stay zeros.
struct Fp8Scale {
  float scale, inv;
};
__device__ __forceinline__ Fp8Scale fp8_scale(float amax) {
  return Fp8Scale{e4m3_row_scale(amax), fminf(e4m3_row_inv(amax), FLT_MAX)};
}

__device__ __forceinline__ float amax8(const float* x) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));   // NaN ignored
  return m;
}

// Eight values times inv to codes, element e in byte e.
__device__ __forceinline__ uint2 fp8_codes8(const float* x, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = pack_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) |
           (pack_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
  return make_uint2(w[0], w[1]);
}

// Two codes of a 16-bit word as fp32 (exact).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t b) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 x;\n\tcvt.rn.f16x2.e4m3x2 x, %2;\n\t"
      "mov.b32 {lo, hi}, x;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y) : "h"((uint16_t)b));
  return f;
}

// Two E2M1 codes of a byte as fp32, the low nibble's first (exact).
__device__ __forceinline__ float2 e2m1x2_to_f32(uint32_t b) {
  uint32_t h;
  asm("{\n\t.reg .b8 t, u;\n\tmov.b16 {t, u}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(h) : "h"((uint16_t)b));
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

__device__ __forceinline__ void unpack8(uint4 v, float* x) {
  x[0] = bf_lo(v.x); x[1] = bf_hi(v.x); x[2] = bf_lo(v.y); x[3] = bf_hi(v.y);
  x[4] = bf_lo(v.z); x[5] = bf_hi(v.z); x[6] = bf_lo(v.w); x[7] = bf_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

}  // namespace farn

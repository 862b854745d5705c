// NVFP4 codes and block scales of a bf16 tensor, and the way back.
//
// The format and the arithmetic are those of farn_forward_nvfp4's copy of
// norm_out (include/farn.h): for tensors that no norm produces -- weights,
// expert activations -- and for reading either kind back.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "farn.h"
#include "farn_internal.h"
#include "farn_kernels.cuh"

using farn_host::DeviceGuard;
using farn_host::overlaps;
using farn_host::product_fits;

namespace {

using farn::bf_hi;
using farn::bf_lo;

constexpr int kThreads = 256;
constexpr int kPerThread = 4;   // blocks of 16 elements per thread, loads in flight

// Two E2M1 codes of a byte as fp32 values, the low nibble's first (exact).
__device__ __forceinline__ float2 e2m1x2_to_f32(uint32_t b) {
  uint32_t h;
  asm("{\n\t.reg .b8 t, u;\n\tmov.b16 {t, u}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(h) : "h"((uint16_t)b));
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// One block of 16 values: scale byte and the 16 codes.  As nvfp4_vec, with
// the block in one thread.
__device__ __forceinline__ uint2 quantize16(const uint32_t* n, float g, uint32_t* sb) {
  float mx = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(n[e])), fabsf(bf_hi(n[e]))));
  const uint32_t s = farn::pack_e4m3x2((mx / 6.0f) * g, 0.0f) & 0xFFu;
  const float sv = farn::e4m3_to_f32(s);
  const float inv = g / sv;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e >> 2] |= farn::pack_e2m1x2(fminf(bf_lo(n[e]) * inv, 6.0f), fminf(bf_hi(n[e]) * inv, 6.0f))
                 << (8 * (e & 3));
  *sb = s;
  return sv > 0.0f ? make_uint2(w[0], w[1]) : make_uint2(0u, 0u);
}

// Memory bound: 2 bytes read and 9/16 written per element.  A row is a
// whole number of blocks and the tensors are contiguous, so the kernel sees
// one array of blocks.  VEC: x 16-byte and codes 8-byte aligned.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const uint16_t* x, uint8_t* codes, uint8_t* scales, float g, int64_t blocks) {
  farn::pdl_wait();
  farn::pdl_trigger();
  const int64_t b0 = (int64_t)blockIdx.x * (kThreads * kPerThread) + threadIdx.x;
  uint32_t n[kPerThread][8];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t b = b0 + i * kThreads;
    if (b >= blocks) continue;
    if constexpr (VEC) {
      const uint4* p = reinterpret_cast<const uint4*>(x + b * 16);
      const uint4 u = farn::ld_stream(p), v = farn::ld_stream(p + 1);
      n[i][0] = u.x; n[i][1] = u.y; n[i][2] = u.z; n[i][3] = u.w;
      n[i][4] = v.x; n[i][5] = v.y; n[i][6] = v.z; n[i][7] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        n[i][e] = (uint32_t)x[b * 16 + 2 * e] | ((uint32_t)x[b * 16 + 2 * e + 1] << 16);
    }
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t b = b0 + i * kThreads;
    if (b >= blocks) continue;
    uint32_t sb;
    const uint2 w = quantize16(n[i], g, &sb);
    if constexpr (VEC) {
      *reinterpret_cast<uint2*>(codes + b * 8) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        codes[b * 8 + e] = (uint8_t)(w.x >> (8 * e));
        codes[b * 8 + 4 + e] = (uint8_t)(w.y >> (8 * e));
      }
    }
    scales[b] = (uint8_t)sb;
  }
}

// value = code * (scale / g), the quotient in fp32, the product rounded to
// bf16.  Memory bound like the other way; a thread takes 8 elements at a time,
// so that a warp's 16-byte stores fill whole lines (16 elements per thread,
// in two stores of half a sector each: 36 us for 8192 x 8192 instead of 26).
// VEC: codes 4-byte and out 16-byte aligned.
constexpr int kHalves = 8;      // half blocks per thread, loads in flight

template <bool VEC>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint8_t* codes, const uint8_t* scales, float g, uint16_t* out,
                  int64_t blocks) {
  farn::pdl_wait();
  farn::pdl_trigger();
  const int64_t halves = blocks * 2;
  const int64_t b0 = (int64_t)blockIdx.x * (kThreads * kHalves) + threadIdx.x;
  uint32_t w[kHalves], sb[kHalves];
#pragma unroll
  for (int i = 0; i < kHalves; ++i) {
    const int64_t b = b0 + i * kThreads;
    if (b >= halves) continue;
    if constexpr (VEC) {
      w[i] = *reinterpret_cast<const uint32_t*>(codes + b * 4);
    } else {
      w[i] = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[i] |= (uint32_t)codes[b * 4 + e] << (8 * e);
    }
    sb[i] = scales[b >> 1];
  }
#pragma unroll
  for (int i = 0; i < kHalves; ++i) {
    const int64_t b = b0 + i * kThreads;
    if (b >= halves) continue;
    const float f = farn::e4m3_to_f32(sb[i]) / g;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = e2m1x2_to_f32((w[i] >> (8 * e)) & 0xFFu);
      o[e] = farn::pack_bf16x2(v.x * f, v.y * f);
    }
    if constexpr (VEC) {
      *reinterpret_cast<uint4*>(out + b * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        out[b * 8 + 2 * e] = (uint16_t)(o[e] & 0xFFFFu);
        out[b * 8 + 2 * e + 1] = (uint16_t)(o[e] >> 16);
      }
    }
  }
}
static_assert(kHalves == 2 * kPerThread, "both kernels take the same number of blocks");

int check_shape(int64_t T, int64_t H, float g) {
  if (T < 0 || H < 1 || H % 16 != 0 || !isfinite(g) || g <= 0.0f) return FARN_ERR_INVALID_ARG;
  if (H > INT64_MAX / 4 || !product_fits(T, 2 * H)) return FARN_ERR_INVALID_ARG;
  return FARN_OK;
}

// Launch over T * H / 16 blocks of 16 elements.
template <typename K, typename... A>
int launch(const farn_ctx* ctx, K kernel, int64_t blocks, cudaStream_t stream, A... args) {
  const int64_t grid = (blocks + kThreads * kPerThread - 1) / (kThreads * kPerThread);
  if (grid > 0x7FFFFFFF) return FARN_ERR_UNSUPPORTED;
  DeviceGuard dg(ctx->device);
  if (!dg.ok) { cudaGetLastError(); return FARN_ERR_CUDA; }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = ctx->pdl ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return FARN_ERR_CUDA;
  }
  return FARN_OK;
}

}  // namespace

extern "C" {

int farn_nvfp4_quantize(const farn_ctx* ctx, const void* x, int64_t T, int64_t H,
                        float tensor_scale, void* codes, void* block_scale,
                        cudaStream_t stream) {
  if (!ctx) return FARN_ERR_INVALID_ARG;
  const int st = check_shape(T, H, tensor_scale);
  if (st != FARN_OK || T == 0) return st;
  if (!x || !codes || !block_scale || ((uintptr_t)x & 1u)) return FARN_ERR_INVALID_ARG;
  const int64_t n = T * H;
  if (overlaps(codes, n / 2, x, n * 2) || overlaps(block_scale, n / 16, x, n * 2) ||
      overlaps(codes, n / 2, block_scale, n / 16))
    return FARN_ERR_ALIAS;
  if (ctx->fault_launch) return FARN_ERR_CUDA;
  const bool vec = ((uintptr_t)x & 15u) == 0 && ((uintptr_t)codes & 7u) == 0 &&
                   ctx->force_variant != kVariantGeneric;
  return launch(ctx, vec ? quantize_kernel<true> : quantize_kernel<false>, n / 16, stream,
                static_cast<const uint16_t*>(x), static_cast<uint8_t*>(codes),
                static_cast<uint8_t*>(block_scale), tensor_scale, n / 16);
}

int farn_nvfp4_dequantize(const farn_ctx* ctx, const void* codes, const void* block_scale,
                          int64_t T, int64_t H, float tensor_scale, void* out,
                          cudaStream_t stream) {
  if (!ctx) return FARN_ERR_INVALID_ARG;
  const int st = check_shape(T, H, tensor_scale);
  if (st != FARN_OK || T == 0) return st;
  if (!codes || !block_scale || !out || ((uintptr_t)out & 1u)) return FARN_ERR_INVALID_ARG;
  const int64_t n = T * H;
  if (overlaps(out, n * 2, codes, n / 2) || overlaps(out, n * 2, block_scale, n / 16))
    return FARN_ERR_ALIAS;
  if (ctx->fault_launch) return FARN_ERR_CUDA;
  const bool vec = ((uintptr_t)out & 15u) == 0 && ((uintptr_t)codes & 3u) == 0 &&
                   ctx->force_variant != kVariantGeneric;
  return launch(ctx, vec ? dequantize_kernel<true> : dequantize_kernel<false>, n / 16, stream,
                static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(block_scale),
                tensor_scale, static_cast<uint16_t*>(out), n / 16);
}

}  // extern "C"

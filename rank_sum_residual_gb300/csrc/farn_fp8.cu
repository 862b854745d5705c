// E4M3 codes and block scales of a bf16 tensor: the operands of the FP8
// products.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "farn.h"
#include "farn_fp8.cuh"
#include "farn_internal.h"

using farn_host::DeviceGuard;
using farn_host::overlaps;
using farn_host::product_fits;

namespace {

constexpr int kThreads = 256;
constexpr int kB = farn::kFp8Block;
constexpr int kLanes = kB / 8;        // lanes of a block's row: 8 elements each
constexpr int kRowBlocks = 4;         // blocks of one row per half warp, loads in flight

// The 8 elements of a row from column h on, as bf16; those outside the row are 0.
// VEC: x 16-byte aligned and H a multiple of 8, so all or none of them exist.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* x, int64_t at, int64_t h, int64_t H) {
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (VEC) {
    if (h < H) u = farn::ld_stream(reinterpret_cast<const uint4*>(x + at));
  } else {
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = h + e < H ? (uint32_t)x[at + e] : 0u;
    u = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
  return u;
}
// The largest magnitudes of two pairs of bf16, NaN ignored.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t amax2(uint4 u) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  return max2(max2(u.x & kAbs, u.y & kAbs), max2(u.z & kAbs, u.w & kAbs));
}
// Of a pair, in fp32; two NaN are 0, as if they had been ignored.
__device__ __forceinline__ float amax_of(uint32_t m) {
  return fmaxf(fmaxf(farn::bf_lo(m), farn::bf_hi(m)), 0.0f);
}
__device__ __forceinline__ uint2 codes8(uint4 u, float inv) {
  float v[8];
  farn::unpack8(u, v);
  return farn::fp8_codes8(v, inv);
}
template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* codes, int64_t at, int64_t h, int64_t H,
                                       uint2 w) {
  if constexpr (VEC) {
    if (h < H) *reinterpret_cast<uint2*>(codes + at) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (h + e < H) codes[at + e] = (uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
  }
}

// Blocks of one row: half a warp each, so that a warp's 8-byte stores fill two
// whole lines.  Memory bound: 2 bytes read and 1 1/32 written per element.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
quantize_rows_kernel(const uint16_t* x, uint8_t* codes, float* scales, int64_t blocks,
                     int64_t HB, int64_t H) {
  farn::pdl_wait();
  farn::pdl_trigger();
  const int lane = threadIdx.x % kLanes, half = threadIdx.x / kLanes;
  constexpr int kHalves = kThreads / kLanes;
  const int64_t b0 = (int64_t)blockIdx.x * (kHalves * kRowBlocks) + half;
  uint4 v[kRowBlocks];
  int64_t at[kRowBlocks], col[kRowBlocks];
#pragma unroll
  for (int i = 0; i < kRowBlocks; ++i) {
    const int64_t b = b0 + i * kHalves;
    const int64_t t = blocks <= 0xFFFFFFFFll ? (int64_t)((uint32_t)b / (uint32_t)HB) : b / HB;
    col[i] = b < blocks ? (b - t * HB) * kB + lane * 8 : H;      // H: no block
    at[i] = t * H + col[i];
    v[i] = load8<VEC>(x, at[i], col[i], H);
  }
#pragma unroll
  for (int i = 0; i < kRowBlocks; ++i) {
    float m = amax_of(amax2(v[i]));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const farn::Fp8Scale s = farn::fp8_scale(m);
    store8<VEC>(codes, at[i], col[i], H, codes8(v[i], s.inv));
    const int64_t b = b0 + i * kHalves;
    if (lane == 0 && b < blocks) scales[b] = s.scale;
  }
}

// Blocks of 128 rows by 128 columns: one per CTA, held in registers between
// its maximum and its codes.  blockIdx.x: (matrix, row block, column block).
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
quantize_tiles_kernel(const uint16_t* x, uint8_t* codes, float* scales, int64_t TB, int64_t HB,
                      int64_t T, int64_t H) {
  __shared__ float warp_max[kThreads / 32];
  farn::pdl_wait();
  farn::pdl_trigger();
  constexpr int kRows = kThreads / kLanes, kPasses = kB / kRows;
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int64_t hb = blockIdx.x % HB, q = blockIdx.x / HB, tb = q % TB, e = q / TB;
  const int64_t h = hb * kB + lane * 8;
  uint4 v[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t t = tb * kB + i * kRows + sub;
    v[i] = load8<VEC>(x, (e * T + t) * H + h, t < T ? h : H, H);
  }
  uint32_t m2 = 0u;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) m2 = max2(m2, amax2(v[i]));
  float m = farn::warp_max(amax_of(m2));
  if (threadIdx.x % 32 == 0) warp_max[threadIdx.x / 32] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, warp_max[w]);
  const farn::Fp8Scale s = farn::fp8_scale(m);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t t = tb * kB + i * kRows + sub;
    store8<VEC>(codes, (e * T + t) * H + h, t < T ? h : H, H, codes8(v[i], s.inv));
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s.scale;
}

template <typename K, typename... A>
int launch(const farn_ctx* ctx, K kernel, int64_t grid, cudaStream_t stream, A... args) {
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

extern "C" int farn_fp8_quantize(const farn_ctx* ctx, const void* x, int64_t E, int64_t T,
                                 int64_t H, int block_rows, void* codes, float* scales,
                                 cudaStream_t stream) {
  if (!ctx || E < 0 || T < 0 || H < 1 || H > INT64_MAX / 4 ||
      (block_rows != 1 && block_rows != kB) || !product_fits(T, 2 * H) ||
      !product_fits(2 * T * H, E))
    return FARN_ERR_INVALID_ARG;
  if (E == 0 || T == 0) return FARN_OK;
  if (!x || !codes || !scales || ((uintptr_t)x & 1u) || ((uintptr_t)scales & 3u))
    return FARN_ERR_INVALID_ARG;
  const int64_t n = E * T * H, HB = (H + kB - 1) / kB, TB = (T + block_rows - 1) / block_rows;
  const int64_t blocks = E * TB * HB;
  if (overlaps(codes, n, x, n * 2) || overlaps(scales, blocks * 4, x, n * 2) ||
      overlaps(codes, n, scales, blocks * 4))
    return FARN_ERR_ALIAS;
  if (ctx->fault_launch) return FARN_ERR_CUDA;
  const bool vec = ((uintptr_t)x & 15u) == 0 && ((uintptr_t)codes & 7u) == 0 && H % 8 == 0 &&
                   ctx->force_variant != kVariantGeneric;
  const uint16_t* in = static_cast<const uint16_t*>(x);
  uint8_t* out = static_cast<uint8_t*>(codes);
  if (block_rows == 1) {
    constexpr int64_t per = (int64_t)(kThreads / kLanes) * kRowBlocks;
    return launch(ctx, vec ? quantize_rows_kernel<true> : quantize_rows_kernel<false>,
                  (blocks + per - 1) / per, stream, in, out, scales, blocks, HB, H);
  }
  return launch(ctx, vec ? quantize_tiles_kernel<true> : quantize_tiles_kernel<false>, blocks,
                stream, in, out, scales, TB, HB, T, H);
}

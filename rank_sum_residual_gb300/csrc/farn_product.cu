// The products: rows by their expert's weights, and NVFP4 by NVFP4.
// Argument checks, the choice of kernel, and the launch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "farn.h"
#include "farn_internal.h"
#include "farn_product.cuh"

static_assert(FARN_MAX_EXPERTS == farn::kMaxExperts, "FARN_MAX_EXPERTS and kernel limit differ");

using farn::ProductParams;
using farn_host::DeviceGuard;
using farn_host::aligned16;
using farn_host::overlaps;
using farn_host::product_fits;

namespace {

typedef void (*ProductKernel)(const ProductParams);

int launch_plain(const farn_ctx* ctx, const ProductParams& p, bool fp4, cudaStream_t stream) {
  // no fewer blocks than tiles for a small call; a long one walks
  const int64_t slot_tiles = p.S / farn::kPlainTile + (p.E < p.S ? p.E : p.S);
  const int64_t tiles =
      slot_tiles * ((p.N + farn::kPlainTile - 1) / farn::kPlainTile);
  const int64_t most = (int64_t)ctx->num_sms * 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles < most ? tiles : most), 1, 1);
  cfg.blockDim = dim3(farn::kPlainThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = ctx->pdl ? 1 : 0;
  ProductKernel k =
      fp4 ? farn::farn_product_plain_kernel<true> : farn::farn_product_plain_kernel<false>;
  if (cudaLaunchKernelEx(&cfg, k, p) != cudaSuccess) {
    cudaGetLastError();
    return FARN_ERR_CUDA;
  }
  return FARN_OK;
}

int launch(const farn_ctx* ctx, const ProductParams& p, bool fp4, cudaStream_t stream) {
  DeviceGuard dg(ctx->device);
  if (!dg.ok) { cudaGetLastError(); return FARN_ERR_CUDA; }
  return launch_plain(ctx, p, fp4, stream);
}

// Slots are 32-bit numbers, and a row of weights fits 31 bits.
bool sizes_ok(int64_t S, int64_t N, int64_t H) {
  return S >= 0 && S <= 0x7FFFFFFF && N >= 1 && N <= 0x7FFFFFFF && H >= 1 && H <= 0x7FFFFFFF &&
         product_fits(S, 2 * N) && product_fits(S, 2 * H);
}

}  // namespace

extern "C" {

int farn_grouped_matmul(const farn_ctx* ctx, const void* x, int64_t n_rows, const int32_t* rows,
                        int64_t n_slots, const void* weights, int E, const int32_t* offsets,
                        int64_t N, int64_t H, void* out, cudaStream_t stream) {
  if (!ctx || n_rows < 0 || n_rows > 0x7FFFFFFF || !sizes_ok(n_slots, N, H) || E < 1 ||
      E > FARN_MAX_EXPERTS || !product_fits(n_rows, 2 * H) || !product_fits(2 * N * H, E) ||
      (!rows && n_rows != n_slots))
    return FARN_ERR_INVALID_ARG;
  if (n_slots == 0) return FARN_OK;
  if ((n_rows > 0 && !x) || !weights || !offsets || !out) return FARN_ERR_INVALID_ARG;
  if (((uintptr_t)x & 1u) || ((uintptr_t)weights & 1u) || ((uintptr_t)out & 1u) ||
      ((uintptr_t)rows & 3u) || ((uintptr_t)offsets & 3u))
    return FARN_ERR_INVALID_ARG;
  const int64_t ob = n_slots * N * 2;
  if (overlaps(out, ob, x, n_rows * H * 2) || overlaps(out, ob, weights, 2 * N * H * E) ||
      overlaps(out, ob, rows, rows ? n_slots * 4 : 0) ||
      overlaps(out, ob, offsets, (int64_t)(E + 1) * 4))
    return FARN_ERR_ALIAS;
  if (ctx->fault_launch) return FARN_ERR_CUDA;
  ProductParams p;
  memset(&p, 0, sizeof p);
  p.a = x;
  p.b = weights;
  p.rows = rows;
  p.offsets = offsets;
  p.out = out;
  p.n_a = n_rows;
  p.S = n_slots;
  p.N = N;
  p.H = H;
  p.E = E;
  p.alpha = 1.0f;
  p.err = ctx->d_status;
  p.stall_test = ctx->stall_test;
  return launch(ctx, p, false, stream);
}

int farn_nvfp4_matmul(const farn_ctx* ctx, const void* a_codes, const void* a_scale,
                      float a_tensor_scale, const void* b_codes, const void* b_scale,
                      float b_tensor_scale, int64_t T, int64_t N, int64_t H, void* out,
                      cudaStream_t stream) {
  if (!ctx || !sizes_ok(T, N, H) || H % 16 != 0 || !product_fits(N, H) ||
      !isfinite(a_tensor_scale) || a_tensor_scale <= 0.0f || !isfinite(b_tensor_scale) ||
      b_tensor_scale <= 0.0f)
    return FARN_ERR_INVALID_ARG;
  if (T == 0) return FARN_OK;
  if (!a_codes || !a_scale || !b_codes || !b_scale || !out || ((uintptr_t)out & 1u))
    return FARN_ERR_INVALID_ARG;
  const int64_t ob = T * N * 2;
  if (overlaps(out, ob, a_codes, T * H / 2) || overlaps(out, ob, a_scale, T * H / 16) ||
      overlaps(out, ob, b_codes, N * H / 2) || overlaps(out, ob, b_scale, N * H / 16))
    return FARN_ERR_ALIAS;
  // 1 / (ga * gb), rounded once; the product of two fp32 values is exact in
  // a double
  const float alpha = (float)(1.0 / ((double)a_tensor_scale * (double)b_tensor_scale));
  if (!isfinite(alpha) || alpha == 0.0f) return FARN_ERR_INVALID_ARG;
  if (ctx->fault_launch) return FARN_ERR_CUDA;
  ProductParams p;
  memset(&p, 0, sizeof p);
  p.a = a_codes;
  p.a_scale = static_cast<const uint8_t*>(a_scale);
  p.b = b_codes;
  p.b_scale = static_cast<const uint8_t*>(b_scale);
  p.out = out;
  p.n_a = T;
  p.S = T;
  p.N = N;
  p.H = H;
  p.E = 1;
  p.alpha = alpha;
  p.err = ctx->d_status;
  p.stall_test = ctx->stall_test;
  return launch(ctx, p, true, stream);
}

}  // extern "C"

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
#include "farn_product_tc.cuh"

static_assert(FARN_MAX_EXPERTS == farn::kMaxExperts, "FARN_MAX_EXPERTS and kernel limit differ");

using farn::ProductParams;
using farn_host::DeviceGuard;
using farn_host::aligned16;
using farn_host::overlaps;
using farn_host::product_fits;

namespace {

typedef void (*ProductKernel)(const ProductParams);

// No more tiles than this: their numbers are 32-bit, with room for a step.
constexpr int64_t kMaxTiles = 0x7FFFFFFF / 2;

int64_t plain_tiles(const ProductParams& p) {
  const int64_t slot_tiles = p.S / farn::kPlainTile + (p.E < p.S ? p.E : p.S);
  return slot_tiles * ((p.N + farn::kPlainTile - 1) / farn::kPlainTile);
}

int launch_plain(const farn_ctx* ctx, const ProductParams& p, bool fp4, cudaStream_t stream) {
  // no fewer blocks than tiles for a small call; a long one walks
  const int64_t tiles = plain_tiles(p);
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

// ------------------------------------------------------ tensor-core kernels
typedef void (*TcKernel)(const farn::TcParams, const CUtensorMap, const CUtensorMap,
                         const CUtensorMap, const CUtensorMap, const CUtensorMap);

struct TcKind {
  bool fp4, gather, copy;
  int cg, bn;
  TcKernel kernel;
  int warps, stage_bytes, scale_bytes, rows, box;
};

template <bool FP4, int CG, int BN, bool GATHER, bool COPY>
TcKind kind() {
  using Sh = farn::TcShape<FP4, CG, BN, GATHER, COPY>;
  return TcKind{FP4, GATHER, COPY, CG, BN,
                &farn::farn_product_tc_kernel<FP4, CG, BN, GATHER, COPY>,
                Sh::kWarps, Sh::kStageBytes, farn::kTcScaleSlots * Sh::kScaleSlot, Sh::kRows, Sh::kBox};
}

const TcKind kKinds[] = {
    kind<false, 1, 64, false, false>(),  kind<false, 1, 64, true, false>(),
    kind<false, 2, 256, false, false>(), kind<false, 2, 256, true, false>(),
    kind<true, 1, 64, false, false>(),   kind<true, 1, 64, false, true>(),
    kind<true, 2, 224, false, false>(),  kind<true, 2, 224, false, true>(),
};

// copy: an NVFP4 call whose block scales TMA cannot read
const TcKind* find_kind(bool fp4, int cg, bool gather, bool copy) {
  for (const TcKind& k : kKinds)
    if (k.fp4 == fp4 && k.cg == cg && k.gather == gather && k.copy == copy)
      return &k;
  return nullptr;
}

struct TcPlan {
  const TcKind* kind;
  int ks, stages;
  unsigned grid;
  uint32_t scales_at, barriers_at, groups_at, part_at, smem;
};

// Shared memory of a call: the ring, the barriers, the groups, and the
// parts that the CTAs of a split row exchange; then 1 KB to align the ring.
bool fit(const farn_ctx* ctx, const TcKind* k, int E, int ks, TcPlan* pl) {
  // the epilogue turns accumulators over, or exchanges parts of a split row
  const uint32_t part =
      ks > 1 ? (uint32_t)k->bn * farn::kPartPitch * 4 : 4 * (uint32_t)farn::kTurnBytes;
  const uint32_t barriers = ((uint32_t)sizeof(farn::TcBarriers) + 15u) / 16 * 16;
  const uint32_t groups = (farn::groups_bytes(E) + 15u) / 16 * 16;
  const uint32_t fixed = 1024 + k->scale_bytes + barriers + groups + part;
  int stages = (ctx->max_smem - (int)fixed) / k->stage_bytes;
  if (stages > farn::kTcMaxStages) stages = farn::kTcMaxStages;
  if (stages < 2 || (k->gather && stages < farn::kTcAuxGather)) return false;
  pl->kind = k;
  pl->ks = ks;
  pl->stages = stages;
  pl->scales_at = (uint32_t)stages * k->stage_bytes;
  pl->barriers_at = pl->scales_at + k->scale_bytes;
  pl->groups_at = pl->barriers_at + barriers;
  pl->part_at = pl->groups_at + groups;
  pl->smem = pl->part_at + part + 1024;
  return true;
}

int log2_of(int v) { return v >= 4 ? 2 : v >= 2 ? 1 : 0; }

// The kernel for a call of S slots in E groups.
bool plan_tc(const farn_ctx* ctx, const ProductParams& p, bool fp4, TcPlan* pl) {
  const bool gather = p.rows != nullptr;
  // TMA reads rows of whole 16-byte pieces
  const bool copy = fp4 && (((uintptr_t)p.a_scale | (uintptr_t)p.b_scale |
                             (uintptr_t)(p.H / 16)) & 15u) != 0;
  const int64_t groups = p.E < p.S ? p.E : p.S;
  const int64_t chunks = (p.H + (fp4 ? 255 : 63)) / (fp4 ? 256 : 64);
  // Slot tiles of `bn`: exact for one group, else every group's rest counted
  // as one more (the offsets are on the device).
  auto tiles_of = [&](int bn, int weights) {
    const int64_t slots = p.E == 1 ? (p.S + bn - 1) / bn : p.S / bn + groups;
    return slots * ((p.N + weights - 1) / weights);
  };
  const TcKind* one = find_kind(fp4, 1, gather, copy);
  const TcKind* pair = find_kind(fp4, 2, gather, copy);
  const int64_t tiles1 = tiles_of(one->bn, farn::kTcWeights);
  const int64_t tiles2 = tiles_of(pair->bn, 2 * farn::kTcWeights);
  if (tiles1 > kMaxTiles || tiles2 > kMaxTiles) return false;
  // One CTA per tile of 128 weights by 64 slots, with the row split over up to
  // four of them, or a pair of CTAs per tile of 256 by 256 (NVFP4: 224):
  // whichever has fewer stages one after the other.  A stage takes much the
  // same time in all of them, as it is bound by its synchronisation (one CTA)
  // or made to be (the pair's tensor work); joining a split row costs about one
  // and a half.  With several groups the number of tiles is an estimate, so the
  // last round of CTAs counts half.  Measured (us, one CTA / pair): NVFP4
  // 8192 x 8192, 8 tokens 13.4 / 14.2, 128 tokens 16.5 / 15.6, 512 tokens 46 /
  // 26; 64 experts 2048 -> 7168 of 16 slots each 274 / 277, of 64 321 / 287, of
  // 256 853 / 365.  Splitting: 30 slots of 32 experts, 5000 -> 1200: 51 whole,
  // 44 by 2, 41 by 4; 512 slots of 64 experts, 2048 -> 7168: 283 whole, 289 by
  // 4.  Clusters of four leave 8 of the 152 SMs out; counting them so changed the
  // choice of 58 in 1500 calls, 21 of which were faster by 5 % and 12 slower.
  // Tiles of 16 and of 32 slots were never faster than of 64 (16 slots each:
  // 304 and 281), tiles of 128 for one CTA hardly, splits by 8 not.
  auto stages_of = [&](int64_t tiles, int64_t at_a_time, double per_tile) {
    const double rounds = (double)tiles / (double)at_a_time;
    if (rounds <= 1.0) return per_tile;
    return (p.E == 1 ? ceil(rounds) : rounds + 0.5) * per_tile;
  };
  auto cost_of_split = [&](int ks) {
    return stages_of(tiles1 * ks, ctx->num_sms,
                     (double)((chunks + ks - 1) / ks) + (ks > 1 ? 1.5 : 0.0));
  };
  int ks = 1;
  for (int k = 2; k <= farn::kTcMaxSplit && chunks >= k * 2; k *= 2)
    if (ctx->max_clusters[log2_of(k)] >= 1 && cost_of_split(k) < cost_of_split(ks)) ks = k;
  if (ctx->tc_split) ks = ctx->tc_split;
  // every CTA has a part of the row, and the device has room for the cluster
  while (ks > 1 && (ks > chunks || ctx->max_clusters[log2_of(ks)] < 1)) ks /= 2;
  const double cost1 = cost_of_split(ks);
  const double cost2 = stages_of(tiles2, ctx->max_clusters[1], (double)chunks);
  bool use_pair = cost2 < cost1 || (cost2 == cost1 && p.S > 32 * groups);
  if (ctx->tc_tile) use_pair = ctx->tc_tile == 256;
  if (use_pair) ks = 1;
  // the parts of a split row take room from the ring: none, if it is short
  const TcKind* k = use_pair ? pair : one;
  if (!fit(ctx, k, p.E, ks, pl) && !fit(ctx, k, p.E, 1, pl)) return false;
  const int csize = use_pair ? 2 : pl->ks;
  const int64_t most = ctx->max_clusters[log2_of(csize)], tiles = use_pair ? tiles2 : tiles1;
  if (most < 1) return false;
  pl->grid = (unsigned)((tiles < most ? tiles : most) * csize);
  return true;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Rows of `inner` elements, `rows` of them, `outer` times (0: a map of two
// dimensions); boxes of 128 bytes by `box` rows, written with the 128-byte
// swizzle, zeros outside the tensor.
bool encode(const farn_ctx* ctx, CUtensorMap* map, bool fp4, const void* base, int64_t inner,
            int64_t rows, int64_t outer, int box) {
  const int64_t bytes = fp4 ? inner / 2 : inner * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)(fp4 ? inner / 2 : inner), (cuuint64_t)rows,
                              (cuuint64_t)(outer ? outer : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)bytes, (cuuint64_t)bytes * (cuuint64_t)rows};
  const cuuint32_t boxes[3] = {fp4 ? 128u : 64u, (cuuint32_t)box, 1u};
  const cuuint32_t steps[3] = {1u, 1u, 1u};
  return ((EncodeTiled)ctx->encode_tiled)(
             map, fp4 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             outer ? 3 : 2, const_cast<void*>(base), dims, strides, boxes, steps,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// Block scales: 64 bytes (1024 elements) of 128 rows, written with the
// 64-byte swizzle.
bool encode_scales(const farn_ctx* ctx, CUtensorMap* map, const void* base, int64_t pitch,
                   int64_t rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)pitch, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t boxes[2] = {(cuuint32_t)farn::kTcScaleRow, 128u};
  const cuuint32_t steps[2] = {1u, 1u};
  return ((EncodeTiled)ctx->encode_tiled)(
             map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes,
             steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// What the tensor-core kernels need of a call: rows that TMA can read (both
// operands 16-byte aligned, rows a multiple of 16 bytes, strides below 2^40)
// and slot numbers with room for a tile behind the last.
bool tc_takes(const farn_ctx* ctx, const ProductParams& p, bool fp4) {
  return ctx->encode_tiled && ctx->force_variant != kVariantGeneric && aligned16(p.a) &&
         aligned16(p.b) && p.H % (fp4 ? 32 : 8) == 0 && p.n_a > 0 && p.S <= 0x7FFFFC00 &&
         p.N <= 0x7FFFFC00 && product_fits(p.N, 2 * p.H) && p.N * 2 * p.H < ((int64_t)1 << 40);
}

int launch_tc(const farn_ctx* ctx, const ProductParams& p, bool fp4, const TcPlan& pl,
              cudaStream_t stream) {
  farn::TcParams t;
  memset(&t, 0, sizeof t);
  t.p = p;
  t.stages = pl.stages;
  t.ks = pl.ks;
  const uint64_t at = (uint64_t)(uintptr_t)p.out | (uint64_t)p.N * 2;   // of every row
  t.store_bytes = at % 16 == 0 ? 16 : at % 8 == 0 ? 8 : 2;
  t.groups_at = pl.groups_at;
  t.scales_at = pl.scales_at;
  t.barriers_at = pl.barriers_at;
  t.part_at = pl.part_at;
  CUtensorMap map_w, map_x, map_part, map_ws, map_xs;
  const TcKind* k = pl.kind;
  if (!encode(ctx, &map_w, fp4, p.b, p.H, p.N, p.E, farn::kTcWeights)) return FARN_ERR_CUDA;
  if (k->gather) {
    map_x = map_part = map_w;     // not read
  } else if (!encode(ctx, &map_x, fp4, p.a, p.H, p.n_a, 0, k->rows)) {
    return FARN_ERR_CUDA;
  } else if (k->box == k->rows) {
    map_part = map_x;
  } else if (!encode(ctx, &map_part, fp4, p.a, p.H, p.n_a, 0, k->box)) {
    return FARN_ERR_CUDA;
  }
  map_ws = map_xs = map_w;        // not read, unless
  if (k->fp4 && !k->copy && (!encode_scales(ctx, &map_ws, p.b_scale, p.H / 16, p.N) ||
                       !encode_scales(ctx, &map_xs, p.a_scale, p.H / 16, p.n_a)))
    return FARN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.grid, 1, 1);
  cfg.blockDim = dim3((unsigned)k->warps * 32, 1, 1);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  unsigned n = 0;
  const unsigned csize = k->cg == 2 ? 2u : (unsigned)pl.ks;
  if (csize > 1) {
    attrs[n].id = cudaLaunchAttributeClusterDimension;
    attrs[n].val.clusterDim.x = csize;
    attrs[n].val.clusterDim.y = 1;
    attrs[n].val.clusterDim.z = 1;
    ++n;
  }
  if (ctx->pdl) {
    attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attrs;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, k->kernel, t, map_w, map_x, map_part, map_ws, map_xs) != cudaSuccess) {
    cudaGetLastError();
    return FARN_ERR_CUDA;
  }
  return FARN_OK;
}

int launch(const farn_ctx* ctx, const ProductParams& p, bool fp4, cudaStream_t stream) {
  TcPlan pl;
  const bool tc = tc_takes(ctx, p, fp4) && plan_tc(ctx, p, fp4, &pl);
  if (!tc && plain_tiles(p) > kMaxTiles) return FARN_ERR_UNSUPPORTED;
  DeviceGuard dg(ctx->device);
  if (!dg.ok) { cudaGetLastError(); return FARN_ERR_CUDA; }
  return tc ? launch_tc(ctx, p, fp4, pl, stream) : launch_plain(ctx, p, fp4, stream);
}

int report_plan(const farn_ctx* ctx, const ProductParams& p, bool fp4, int* variant, int* ctas,
                int* threads) {
  TcPlan pl;
  if (tc_takes(ctx, p, fp4) && plan_tc(ctx, p, fp4, &pl)) {
    *variant = pl.kind->cg == 2 ? kVariantPair : kVariantTensor;
    *ctas = pl.kind->cg == 2 ? 2 : pl.ks;
    *threads = pl.kind->warps * 32;
  } else if (plain_tiles(p) > kMaxTiles) {
    return FARN_ERR_UNSUPPORTED;
  } else {
    *variant = kVariantGeneric;
    *ctas = 1;
    *threads = farn::kPlainThreads;
  }
  return FARN_OK;
}

// Slots are 32-bit numbers, and a row of weights fits 31 bits.
bool sizes_ok(int64_t S, int64_t N, int64_t H) {
  return S >= 0 && S <= 0x7FFFFFFF && N >= 1 && N <= 0x7FFFFFFF && H >= 1 && H <= 0x7FFFFFFF &&
         product_fits(S, 2 * N) && product_fits(S, 2 * H);
}

}  // namespace

namespace farn_host {

// On the current device: the tensor-map encoder, the kernels' shared-memory
// opt-in, and how many clusters of one-per-SM CTAs fit at a time.
bool product_setup(farn_ctx* ctx) {
  ctx->encode_tiled = nullptr;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return false;
  for (const TcKind& k : kKinds)
    if (cudaFuncSetAttribute((const void*)k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ctx->max_smem) != cudaSuccess)
      return false;
  for (int i = 0; i < 3; ++i) {
    // one CTA per SM, as any of the kernels takes it
    const TcKind* k = find_kind(false, 1, false, false);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(1 << i), 1, 1);
    cfg.blockDim = dim3((unsigned)k->warps * 32, 1, 1);
    cfg.dynamicSmemBytes = ctx->max_smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << i;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&ctx->max_clusters[i], (const void*)k->kernel, &cfg) !=
            cudaSuccess ||
        (i < 2 && ctx->max_clusters[i] < 1))
      return false;
  }
  ctx->encode_tiled = fn;
  return true;
}

}  // namespace farn_host

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

int farn_plan_grouped_matmul(const farn_ctx* ctx, const void* x, int64_t n_rows,
                             const int32_t* rows, int64_t n_slots, const void* weights, int E,
                             int64_t N, int64_t H, const void* out, int* variant, int* ctas,
                             int* threads) {
  if (!ctx || !variant || !ctas || !threads || n_rows < 0 || n_rows > 0x7FFFFFFF ||
      !sizes_ok(n_slots, N, H) || n_slots < 1 || E < 1 || E > FARN_MAX_EXPERTS ||
      !product_fits(n_rows, 2 * H) || !product_fits(2 * N * H, E) ||
      (!rows && n_rows != n_slots) || !weights || !out)
    return FARN_ERR_INVALID_ARG;
  ProductParams p;
  memset(&p, 0, sizeof p);
  p.a = x;
  p.b = weights;
  p.rows = rows;
  p.out = const_cast<void*>(out);
  p.n_a = n_rows;
  p.S = n_slots;
  p.N = N;
  p.H = H;
  p.E = E;
  return report_plan(ctx, p, false, variant, ctas, threads);
}

int farn_plan_nvfp4_matmul(const farn_ctx* ctx, const void* a_codes, const void* a_scale,
                           const void* b_codes, const void* b_scale, int64_t T, int64_t N,
                           int64_t H, const void* out, int* variant, int* ctas, int* threads) {
  if (!ctx || !variant || !ctas || !threads || !sizes_ok(T, N, H) || T < 1 || H % 16 != 0 ||
      !product_fits(N, H) || !a_codes || !a_scale || !b_codes || !b_scale || !out)
    return FARN_ERR_INVALID_ARG;
  ProductParams p;
  memset(&p, 0, sizeof p);
  p.a = a_codes;
  p.a_scale = static_cast<const uint8_t*>(a_scale);
  p.b = b_codes;
  p.b_scale = static_cast<const uint8_t*>(b_scale);
  p.out = const_cast<void*>(out);
  p.n_a = T;
  p.S = T;
  p.N = N;
  p.H = H;
  p.E = 1;
  return report_plan(ctx, p, true, variant, ctas, threads);
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

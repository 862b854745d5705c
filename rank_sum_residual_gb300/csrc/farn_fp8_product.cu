// The FP8 products with block scales, dense and by expert: argument checks,
// the choice of kernel, and the launch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "farn.h"
#include "farn_fp8_product.cuh"
#include "farn_internal.h"

using farn::Fp8Params;
using farn::ProductParams;
using farn_host::DeviceGuard;
using farn_host::aligned16;
using farn_host::overlaps;
using farn_host::product_fits;

namespace {

// No more tiles than this: their numbers are 32-bit, with room for a step.
constexpr int64_t kMaxTiles = 0x7FFFFFFF / 2;

typedef void (*Kernel)(const Fp8Params, const CUtensorMap, const CUtensorMap);

struct Kind {
  bool gather;
  int cg, bn, warps, regs;
  Kernel kernel;
  int stage_bytes, scale_bytes, part_bytes;
};

template <typename Sh>
Kind kind(bool gather, Kernel kernel) {
  return Kind{gather, Sh::kCg, Sh::kBn, Sh::kWarps, Sh::kRegs, kernel, Sh::kStageBytes,
              Sh::kScaleBytes, Sh::kPartBytes};
}

const Kind kKinds[] = {kind<farn::Fp8One<false>>(false, farn::farn_fp8_one_kernel<false>),
                       kind<farn::Fp8One<true>>(true, farn::farn_fp8_one_kernel<true>),
                       kind<farn::Fp8Pair>(false, farn::farn_fp8_pair_kernel)};

const Kind* find_kind(int cg, bool gather) {
  for (const Kind& k : kKinds)
    if (k.cg == cg && k.gather == gather) return &k;
  return nullptr;
}

struct Plan {
  const Kind* kind;
  int ks, stages;
  unsigned grid;
  uint32_t scales_at, barriers_at, groups_at, part_at, smem;
};

int64_t plain_tiles(const ProductParams& p) {
  const int64_t slot_tiles = p.S / farn::kPlainTile + (p.E < p.S ? p.E : p.S);
  return slot_tiles * ((p.N + farn::kPlainTile - 1) / farn::kPlainTile);
}

int log2_of(int v) { return v >= 4 ? 2 : v >= 2 ? 1 : 0; }

// Shared memory of a call: the ring, the scales, the barriers, the groups, and
// the parts that the CTAs of a split row exchange (or where the adding warps
// turn their sums over); then 1 KB to align the ring.
bool fit(const farn_ctx* ctx, const Kind* k, int E, int ks, Plan* pl) {
  const uint32_t part = ks > 1 ? (uint32_t)k->bn * farn::kPartPitch * 4 : (uint32_t)k->part_bytes;
  const uint32_t barriers = ((uint32_t)sizeof(farn::Fp8Barriers) + 15u) / 16 * 16;
  const uint32_t groups = (farn::groups_bytes(E) + 15u) / 16 * 16;
  const uint32_t fixed = 1024 + k->scale_bytes + barriers + groups + part;
  int stages = (ctx->max_smem - (int)fixed) / k->stage_bytes;
  if (stages > farn::kTcMaxStages) stages = farn::kTcMaxStages;
  if (stages < 2 || (k->gather && stages <= farn::kF8Gather)) return false;
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

// The kernel for a call of S slots in E groups: whichever of one CTA per tile,
// splitting the row or not, and a pair of CTAs has less to do one after the other,
// counted in the one CTA's stages of 0.26 us.  A pair's takes 0.42 us; joining a
// split row 2 us with few slots and twice that with a full tile.  With several
// groups the number of tiles is an estimate, so the last round of CTAs counts
// half.  Measured (us: one CTA, row split by 2, by 4, pair): 1 x 8192 x 8192 20.3,
// 18.4, 19.3, 29.2; 64 x 8192 x 8192 22.3, 19.3, 22.5, 30.0; 100 x 8192 x 8192 23.4,
// 28.7, 35.2, 30.1; 128 x 10240 x 5120 27.4, 30.7, 35.8, 22.9; 400 x 8192 x 2048
// 19.9, 35.9, 57.9, 14.2; 700 x 1000 x 8192 22.2, 27.3, 26.5, 29.7; 64 experts of 64
// slots 2048 -> 4096 114, 235, 392, 126, of 250 4096 -> 2048 353, 517, 757, 183.
//
// can_copy: gathered rows can be laid side by side first, as the pair needs them.
bool plan_tc(const farn_ctx* ctx, const ProductParams& p, bool can_copy, Plan* pl) {
  const bool gather = p.rows != nullptr;
  const int64_t groups = p.E < p.S ? p.E : p.S;
  const int64_t chunks = (p.H + farn::kTcRowBytes - 1) / farn::kTcRowBytes;
  auto tiles_of = [&](int bn, int weights) {
    const int64_t slots = p.E == 1 ? (p.S + bn - 1) / bn : p.S / bn + groups;
    return slots * ((p.N + weights - 1) / weights);
  };
  const Kind* one = find_kind(1, gather);
  const Kind* pair = find_kind(2, false);
  const int64_t tiles1 = tiles_of(one->bn, farn::kTcWeights);
  const int64_t tiles2 = tiles_of(pair->bn, 2 * farn::kTcWeights);
  if (tiles1 > kMaxTiles || tiles2 > kMaxTiles) return false;
  auto stages_of = [&](int64_t tiles, int64_t at_a_time, double per_tile) {
    const double rounds = (double)tiles / (double)at_a_time;
    if (rounds <= 1.0) return per_tile;
    return (p.E == 1 ? ceil(rounds) : rounds + 0.5) * per_tile;
  };
  const double fill = (double)p.S / (double)(groups * one->bn);
  const double join = 7.5 * (1.0 + (fill < 1.0 ? fill : 1.0));
  auto cost_of_split = [&](int ks) {
    return stages_of(tiles1 * ks, ctx->num_sms,
                     (double)((chunks + ks - 1) / ks) + (ks > 1 ? join : 0.0));
  };
  int ks = 1;
  for (int k = 2; k <= farn::kTcMaxSplit && chunks >= k; k *= 2)
    if (ctx->max_clusters[log2_of(k)] >= 1 && cost_of_split(k) < cost_of_split(ks)) ks = k;
  if (ctx->tc_split) ks = ctx->tc_split;
  // every CTA has a part of the row, and the device has room for the cluster
  while (ks > 1 && (ks > chunks || ctx->max_clusters[log2_of(ks)] < 1)) ks /= 2;
  const double cost1 = cost_of_split(ks);
  const double cost2 = 1.65 * stages_of(tiles2, ctx->max_clusters[1], (double)chunks);
  bool use_pair = cost2 < cost1;
  if (ctx->tc_tile) use_pair = ctx->tc_tile == 256;
  if (gather && !can_copy) use_pair = false;
  if (use_pair) ks = 1;
  // the parts of a split row take room from the ring: none, if it is short
  const Kind* k = use_pair ? pair : one;
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

// Rows of H codes, `rows` of them, `outer` times (0: a map of two dimensions);
// boxes of 128 bytes by `box` rows, written with the 128-byte swizzle, zeros
// outside the tensor.
bool encode(const farn_ctx* ctx, CUtensorMap* map, const void* base, int64_t H, int64_t rows,
            int64_t outer, int box) {
  const cuuint64_t dims[3] = {(cuuint64_t)H, (cuuint64_t)rows, (cuuint64_t)(outer ? outer : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)H, (cuuint64_t)H * (cuuint64_t)rows};
  const cuuint32_t boxes[3] = {(cuuint32_t)farn::kTcRowBytes, (cuuint32_t)box, 1u};
  const cuuint32_t steps[3] = {1u, 1u, 1u};
  return ((EncodeTiled)ctx->encode_tiled)(
             map, CU_TENSOR_MAP_DATA_TYPE_UINT8, outer ? 3 : 2, const_cast<void*>(base), dims,
             strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// What the tensor-core kernels need of a call: rows that TMA can read (both
// operands 16-byte aligned, rows a multiple of 16 bytes, strides below 2^40)
// and slot numbers with room for a tile behind the last.
bool tc_takes(const farn_ctx* ctx, const ProductParams& p) {
  return ctx->fp8_ok && ctx->force_variant != kVariantGeneric && aligned16(p.a) &&
         aligned16(p.b) && p.H % 16 == 0 && p.n_a > 0 && p.S <= 0x7FFFFC00 &&
         p.N <= 0x7FFFFC00 && product_fits(p.N, p.H) && p.N * p.H < ((int64_t)1 << 40);
}

template <typename... A>
int launch_kernel(const farn_ctx* ctx, void (*kernel)(A...), unsigned grid, unsigned threads,
                  uint32_t smem, unsigned csize, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  unsigned n = 0;
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
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return FARN_ERR_CUDA;
  }
  return FARN_OK;
}

// Where the rows of a gathering call are laid side by side: codes, then scales.
int64_t copied_codes(int64_t S, int64_t H) { return (S * H + 15) / 16 * 16; }

int launch(const farn_ctx* ctx, Fp8Params t, void* workspace, cudaStream_t stream) {
  ProductParams& p = t.p;
  Plan pl;
  const bool tc = tc_takes(ctx, p) && plan_tc(ctx, p, workspace != nullptr, &pl);
  const int64_t tiles = plain_tiles(p);
  if (!tc && tiles > kMaxTiles) return FARN_ERR_UNSUPPORTED;
  DeviceGuard dg(ctx->device);
  if (!dg.ok) { cudaGetLastError(); return FARN_ERR_CUDA; }
  if (!tc) {
    const int64_t most = (int64_t)ctx->num_sms * 4;
    return launch_kernel(ctx, farn::farn_fp8_product_plain_kernel,
                         (unsigned)(tiles < most ? tiles : most), farn::kPlainThreads, 0, 1,
                         stream, t);
  }
  const bool copy = p.rows && pl.kind->cg == 2;
  farn::Fp8GatherParams g;
  if (copy) {
    g = {static_cast<const uint8_t*>(p.a), t.a_scale, p.rows, static_cast<uint8_t*>(workspace),
         reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + copied_codes(p.S, p.H)),
         p.n_a, p.S, p.H, t.HB};
    t.n_rows = p.n_a;
    p.a = g.to;
    t.a_scale = g.to_scale;
    p.n_a = p.S;
  }
  t.stages = pl.stages;
  t.ks = pl.ks;
  const uint64_t at = (uint64_t)(uintptr_t)p.out | (uint64_t)p.N * 2;   // of every row
  t.store_bytes = at % 16 == 0 ? 16 : at % 8 == 0 ? 8 : 2;
  t.scale_vec = t.HB % 4 == 0 && aligned16(t.a_scale) && aligned16(t.b_scale);
  t.scales_at = pl.scales_at;
  t.barriers_at = pl.barriers_at;
  t.groups_at = pl.groups_at;
  t.part_at = pl.part_at;
  const Kind* k = pl.kind;
  CUtensorMap map_w, map_x;
  if (!encode(ctx, &map_w, p.b, p.H, p.N, p.E, 64)) return FARN_ERR_CUDA;
  map_x = map_w;                    // not read, unless
  if (!k->gather && !encode(ctx, &map_x, p.a, p.H, p.n_a, 0, farn::kF8Box)) return FARN_ERR_CUDA;
  if (copy) {
    constexpr int64_t per = farn::kF8CopyThreads / 32;
    const int st = launch_kernel(ctx, farn::fp8_gather_kernel, (unsigned)((p.S + per - 1) / per),
                                 farn::kF8CopyThreads, 0, 1, stream, g);
    if (st != FARN_OK) return st;
  }
  return launch_kernel(ctx, k->kernel, pl.grid, k->warps * 32u, pl.smem,
                       k->cg == 2 ? 2u : (unsigned)pl.ks, stream, t, map_w, map_x);
}

int report_plan(const farn_ctx* ctx, const ProductParams& p, bool can_copy, int* variant,
                int* ctas, int* threads) {
  Plan pl;
  if (tc_takes(ctx, p) && plan_tc(ctx, p, can_copy, &pl)) {
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

int64_t blocks_of(int64_t n) { return (n + farn::kFp8Block - 1) / farn::kFp8Block; }

}  // namespace

namespace farn_host {

// On the current device, after product_setup: the kernels' shared-memory opt-in.
// The pairs' kernels hand registers from some warps to others, and a launch with
// fewer than they share out would wait for ever: none is made then.
bool fp8_product_setup(const farn_ctx* ctx) {
  for (const Kind& k : kKinds) {
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, (const void*)k.kernel) != cudaSuccess ||
        attr.numRegs < k.regs ||
        cudaFuncSetAttribute((const void*)k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ctx->max_smem) != cudaSuccess)
      return false;
  }
  return true;
}

}  // namespace farn_host

extern "C" {

int farn_fp8_matmul(const farn_ctx* ctx, const void* a_codes, const float* a_scale,
                    const void* b_codes, const float* b_scale, int64_t T, int64_t N, int64_t H,
                    void* out, cudaStream_t stream) {
  if (!ctx || !sizes_ok(T, N, H) || !product_fits(N, H)) return FARN_ERR_INVALID_ARG;
  if (T == 0) return FARN_OK;
  if (!a_codes || !a_scale || !b_codes || !b_scale || !out || ((uintptr_t)out & 1u) ||
      (((uintptr_t)a_scale | (uintptr_t)b_scale) & 3u))
    return FARN_ERR_INVALID_ARG;
  const int64_t HB = blocks_of(H), NB = blocks_of(N), ob = T * N * 2;
  if (overlaps(out, ob, a_codes, T * H) || overlaps(out, ob, a_scale, T * HB * 4) ||
      overlaps(out, ob, b_codes, N * H) || overlaps(out, ob, b_scale, NB * HB * 4))
    return FARN_ERR_ALIAS;
  if (ctx->fault_launch) return FARN_ERR_CUDA;
  Fp8Params t;
  memset(&t, 0, sizeof t);
  t.p.a = a_codes;
  t.p.b = b_codes;
  t.p.out = out;
  t.p.n_a = T;
  t.p.S = T;
  t.p.N = N;
  t.p.H = H;
  t.p.E = 1;
  t.p.alpha = 1.0f;
  t.p.err = ctx->d_status;
  t.p.stall_test = ctx->stall_test;
  t.a_scale = a_scale;
  t.b_scale = b_scale;
  t.HB = HB;
  t.NB = NB;
  return launch(ctx, t, nullptr, stream);
}

int farn_plan_fp8_matmul(const farn_ctx* ctx, const void* a_codes, const void* b_codes, int64_t T,
                         int64_t N, int64_t H, const void* out, int* variant, int* ctas,
                         int* threads) {
  if (!ctx || !variant || !ctas || !threads || !sizes_ok(T, N, H) || T < 1 || !product_fits(N, H) ||
      !a_codes || !b_codes || !out)
    return FARN_ERR_INVALID_ARG;
  ProductParams p;
  memset(&p, 0, sizeof p);
  p.a = a_codes;
  p.b = b_codes;
  p.n_a = T;
  p.S = T;
  p.N = N;
  p.H = H;
  p.E = 1;
  return report_plan(ctx, p, false, variant, ctas, threads);
}

int farn_plan_fp8_grouped_matmul(const farn_ctx* ctx, const void* x, int64_t n_rows,
                                 const int32_t* rows, int64_t n_slots, const void* weights, int E,
                                 int64_t N, int64_t H, const void* out, const void* workspace,
                                 int* variant, int* ctas, int* threads) {
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
  p.n_a = n_rows;
  p.S = n_slots;
  p.N = N;
  p.H = H;
  p.E = E;
  return report_plan(ctx, p, workspace && aligned16(workspace), variant, ctas, threads);
}

int farn_fp8_grouped_workspace(const farn_ctx* ctx, int64_t n_slots, int E, int64_t N, int64_t H,
                               int64_t* bytes) {
  if (!ctx || !bytes || !sizes_ok(n_slots, N, H) || E < 1 || E > FARN_MAX_EXPERTS)
    return FARN_ERR_INVALID_ARG;
  *bytes = 0;
  if (n_slots == 0 || H % 16 != 0 || !ctx->fp8_ok || ctx->force_variant == kVariantGeneric)
    return FARN_OK;
  // what plan_tc goes by: sizes, and that the rows are gathered
  static const int32_t some_rows = 0;
  ProductParams p;
  memset(&p, 0, sizeof p);
  p.rows = &some_rows;
  p.S = n_slots;
  p.N = N;
  p.H = H;
  p.E = E;
  Plan pl;
  if (plan_tc(ctx, p, true, &pl) && pl.kind->cg == 2)
    *bytes = copied_codes(n_slots, H) + n_slots * blocks_of(H) * 4;
  return FARN_OK;
}

int farn_fp8_grouped_matmul(const farn_ctx* ctx, const void* x, const float* x_scale,
                            int64_t n_rows, const int32_t* rows, int64_t n_slots,
                            const void* weights, const float* w_scale, int E,
                            const int32_t* offsets, int64_t N, int64_t H, void* out,
                            void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  if (!ctx || workspace_bytes < 0 || n_rows < 0 || n_rows > 0x7FFFFFFF ||
      !sizes_ok(n_slots, N, H) || E < 1 || E > FARN_MAX_EXPERTS ||
      !product_fits(n_rows, 2 * H) || !product_fits(2 * N * H, E) ||
      (!rows && n_slots > 0 && n_rows != n_slots))
    return FARN_ERR_INVALID_ARG;
  if (n_slots == 0) return FARN_OK;
  if ((n_rows > 0 && (!x || !x_scale)) || !weights || !w_scale || !offsets || !out)
    return FARN_ERR_INVALID_ARG;
  if (((uintptr_t)out & 1u) || (((uintptr_t)rows | (uintptr_t)offsets | (uintptr_t)x_scale |
                                 (uintptr_t)w_scale) & 3u))
    return FARN_ERR_INVALID_ARG;
  const int64_t HB = blocks_of(H), NB = blocks_of(N), ob = n_slots * N * 2;
  if (overlaps(out, ob, x, n_rows * H) || overlaps(out, ob, x_scale, n_rows * HB * 4) ||
      overlaps(out, ob, weights, N * H * E) || overlaps(out, ob, w_scale, NB * HB * E * 4) ||
      overlaps(out, ob, rows, rows ? n_slots * 4 : 0) ||
      overlaps(out, ob, offsets, (int64_t)(E + 1) * 4))
    return FARN_ERR_ALIAS;
  // the workspace: used if it is given, large enough and aligned
  const int64_t need = copied_codes(n_slots, H) + n_slots * HB * 4;
  if (!rows || !workspace || !aligned16(workspace) || workspace_bytes < need) workspace = nullptr;
  if (workspace &&
      (overlaps(workspace, need, out, ob) || overlaps(workspace, need, x, n_rows * H) ||
       overlaps(workspace, need, x_scale, n_rows * HB * 4) ||
       overlaps(workspace, need, weights, N * H * E) ||
       overlaps(workspace, need, w_scale, NB * HB * E * 4) ||
       overlaps(workspace, need, rows, n_slots * 4) ||
       overlaps(workspace, need, offsets, (int64_t)(E + 1) * 4)))
    return FARN_ERR_ALIAS;
  if (ctx->fault_launch) return FARN_ERR_CUDA;
  Fp8Params t;
  memset(&t, 0, sizeof t);
  t.p.a = x;
  t.p.b = weights;
  t.p.rows = rows;
  t.p.offsets = offsets;
  t.p.out = out;
  t.p.n_a = n_rows;
  t.p.S = n_slots;
  t.p.N = N;
  t.p.H = H;
  t.p.E = E;
  t.p.alpha = 1.0f;
  t.p.err = ctx->d_status;
  t.p.stall_test = ctx->stall_test;
  t.a_scale = x_scale;
  t.b_scale = w_scale;
  t.HB = HB;
  t.NB = NB;
  return launch(ctx, t, workspace, stream);
}

}  // extern "C"

// The FP8 products: E4M3 codes with an fp32 scale for every 128 elements of a
// slot's row and every 128 x 128 of the weights.
//
//     out[s, n] = sum_b (sa[s, b] * sb[n / 128, b]) * sum_{h in b} a[s, h] * b[n, h]
//
// The inner sums are matrix instructions over one block's 128 bytes of a row
// (one stage of the ring); the outer sum is fp32 multiply-adds in registers,
// because the matrix instructions know scales of blocks of 32 with powers of
// two only.  Each block's sums are handed to eight adding warps through tensor
// memory, which holds the sums of two blocks (`one`: four).
//
//   pair    a pair of CTAs per tile of 256 slots by 256 weights: long calls.
//           The slots are the matrix instruction's M side, so a lane has one
//           slot and an adding warp one block of weights: a block's factor sa *
//           sb is one value per lane.  Halves of 128 weights are handed over by
//           themselves: one is read while the other three are computed.
//   one     a CTA per tile of 128 weights (the M side) by 64 slots: short
//           calls, where a tile of slots is mostly empty.  A slot's factor is a
//           column's and comes from shared memory.  Up to four CTAs of a cluster
//           split the row and join their sums, in rank order, through
//           distributed shared memory.
//
// Warps of a CTA: eight that add and store; one or two that have TMA fetch the
// weights and the slots' rows, or (`one`) four that copy gathered rows themselves;
// one (`pair`: for each half one) that issues the matrix instructions; one that
// fetches the scales and leaves the products sa * sb in shared memory.
//
// Every wait is bounded (see tc_wait).
#pragma once

#include <cuda.h>

#include "farn_fp8.cuh"
#include "farn_product_tc.cuh"

namespace farn {

constexpr int kF8Adders = 8;           // warps
constexpr int kF8Box = 32;             // slots' rows of a TMA box
constexpr int kF8ScaleBlocks = 4;      // blocks of a row whose scales are fetched together
constexpr int kF8ScaleSlots = 3;       // such groups in shared memory
constexpr int kF8Gather = 4;           // warps; not more than the ring has stages

struct Fp8Params {
  ProductParams p;                     // a, b: E4M3 codes
  const float* a_scale;                // [n_a, HB]
  const float* b_scale;                // [E, NB, HB]
  int64_t HB, NB;
  int64_t n_rows;                      // `pair` of gathered rows: what the rows index
  int scale_vec;                       // the scales' rows can be read 16 bytes at a time
  int stages;
  int ks;                              // `one`: CTAs of a cluster that split the row
  int store_bytes;                     // 16, 8 or 2: what N and out allow a store to be
  uint32_t scales_at, barriers_at, groups_at, part_at;   // shared-memory offsets
};

struct Fp8Barriers {
  uint64_t full[kTcMaxStages];
  uint64_t empty[kTcMaxStages];
  uint64_t acc_full[4];                // [buffer][half]
  uint64_t acc_empty[4];
  uint64_t scale_full[kF8ScaleSlots];
  uint64_t scale_empty[kF8ScaleSlots];
  uint64_t part_full;
  uint64_t part_empty;
  uint64_t never;
  uint32_t tmem;
  int abort_flag;
};

struct Fp8Pair {
  static constexpr int kCg = 2;
  static constexpr int kBn = 256;                         // slots of a tile
  static constexpr int kTileWeights = 256;
  static constexpr int kHalf = 128;                       // weights that are handed over alone
  static constexpr int kWarps = 12;
  // Registers of a thread at launch, and once the adding warps have taken some
  // from the others (setmaxnreg): the shares add up to what the launch gave.
  static constexpr int kRegs = 168, kAddRegs = 216, kRestRegs = 72;
  static_assert(kAddRegs * kF8Adders + kRestRegs * (kWarps - kF8Adders) <= kRegs * kWarps, "");
  static constexpr int kSlotBytes = 128 * kTcRowBytes;    // of a stage, per CTA
  static constexpr int kStageBytes = 2 * kSlotBytes;
  // of a group of blocks: a factor per block, half of the weights, and slot
  static constexpr int kScaleSlot = kF8ScaleBlocks * 2 * 128 * 4;
  static constexpr int kScaleBytes = kF8ScaleSlots * kScaleSlot;
  static constexpr int kCols = 512;
  static constexpr int kPartBytes = kF8Adders * 32 * 80;  // see store_rows
};
template <bool GATHER>
struct Fp8One {
  static constexpr int kCg = 1;
  static constexpr int kBn = 64;                          // slots of a tile
  static constexpr int kTileWeights = 128;
  static constexpr int kWarps = GATHER ? 16 : 12;
  static constexpr int kRegs = 0;
  static constexpr int kWarpCols = kBn / 2;               // columns of an adding warp
  static constexpr int kABytes = kTcWeights * kTcRowBytes;
  static constexpr int kStageBytes = kABytes + kBn * kTcRowBytes;
  static constexpr int kScaleSlot = kF8ScaleBlocks * kBn * 4;
  static constexpr int kScaleBytes = kF8ScaleSlots * kScaleSlot;
  static constexpr int kBufs = 4;                         // blocks' sums in tensor memory
  static constexpr int kCols = kBufs * kBn;
  static constexpr int kPartBytes = kF8Adders * kTurnBytes;
};

// d += v * s for two values each, s twice the same; one rounding per value.  (Single
// multiply-adds took 1 to 2 % longer.)
__device__ __forceinline__ void fma_pair(uint64_t& d, uint32_t v0, uint32_t v1, uint64_t s) {
  asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
      : "+l"(d) : "r"(v0), "r"(v1), "l"(s));
}
__device__ __forceinline__ uint64_t twice(float s) {
  return ((uint64_t)__float_as_uint(s) << 32) | __float_as_uint(s);
}

// What a wait orders.  kOwn: the CTA's own threads (and TMA, and the matrix
// instructions) arrive on the barrier.  kCluster: another CTA of the pair too, and
// what it did to shared memory is ordered before what follows.  kTensor: tensor
// memory alone is handed over, which the tcgen05 fences on both sides order: the
// arrivals and the wait are relaxed, at the cluster's scope.
enum Fp8Wait { kOwn, kCluster, kTensor };

// Whether a phase is complete: test_wait (LOOK) says so at once, try_wait may let
// the thread sleep first.
template <Fp8Wait WHAT, bool LOOK>
__device__ __forceinline__ uint32_t f8_phase(uint32_t bar, uint32_t parity) {
  uint32_t ok;
#define FARN_F8_PHASE(form)                                                             \
  asm volatile("{\n\t.reg .pred p;\n\t" form " p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}" \
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory")
  if constexpr (WHAT == kTensor) {
    if constexpr (LOOK) FARN_F8_PHASE("mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64");
    else FARN_F8_PHASE("mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64");
  } else if constexpr (WHAT == kCluster) {
    if constexpr (LOOK) FARN_F8_PHASE("mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64");
    else FARN_F8_PHASE("mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64");
  } else {
    if constexpr (LOOK) FARN_F8_PHASE("mbarrier.test_wait.parity.shared::cta.b64");
    else FARN_F8_PHASE("mbarrier.try_wait.parity.shared::cta.b64");
  }
#undef FARN_F8_PHASE
  return ok;
}

// A warp's wait as tc_wait_warp, with a short way for a phase that is complete:
// the general one takes 150 to 200 cycles even then.
template <Fp8Wait WHAT>
__device__ __forceinline__ bool f8_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                        int* err, int code) {
  if (__all_sync(0xFFFFFFFFu, f8_phase<WHAT, false>(bar, parity))) return true;
  return tc_wait_warp<WHAT != kOwn>(bar, parity, abort_flag, err, code);
}
// The same in two halves: a look ahead, whose answer is not needed yet, and the
// wait that it may save.  (A try_wait in place of the look held up what stood
// between the two: 8192^3 421 us instead of 415.)
template <Fp8Wait WHAT>
__device__ __forceinline__ uint32_t f8_look(uint32_t bar, uint32_t parity) {
  return f8_phase<WHAT, true>(bar, parity);
}
template <Fp8Wait WHAT>
__device__ __forceinline__ bool f8_answer(uint32_t looked, uint32_t bar, uint32_t parity,
                                          volatile int* abort_flag, int* err, int code) {
  if (__all_sync(0xFFFFFFFFu, looked)) return true;
  return f8_wait<WHAT>(bar, parity, abort_flag, err, code);
}

// Arrive on the first CTA's barrier for reads of tensor memory that are done
// (tcgen05.wait::ld): nothing in ordinary memory is handed over with it, so the
// arrival has no release, which would cost the warp about 150 cycles.
// By one lane, without a branch.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr, int lane) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t"
               "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}"
               :: "r"(cluster_addr), "r"(lane) : "memory");
}
// On a barrier of the own CTA, by one lane.
__device__ __forceinline__ void arrive_local(uint32_t bar, int lane) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t"
               "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}"
               :: "r"(bar), "r"(lane) : "memory");
}

// The scales of kF8ScaleBlocks blocks of a row from block c on, those from
// `end` on 0; row null: 0.
__device__ __forceinline__ float4 load_scales(const float* row, int c, int end, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!row) return v;
  if (vec && c + kF8ScaleBlocks <= end && (c & 3) == 0)
    return __ldg(reinterpret_cast<const float4*>(row + c));
  if (c < end) v.x = __ldg(row + c);
  if (c + 1 < end) v.y = __ldg(row + c + 1);
  if (c + 2 < end) v.z = __ldg(row + c + 2);
  if (c + 3 < end) v.w = __ldg(row + c + 3);
  return v;
}

// 32 columns of a warp's 32 rows, from a row per lane to the output: turned in
// shared memory (rows of 80 bytes: 16-byte accesses without bank conflicts) and
// written in runs of 64 bytes.  rows: those that exist; col: the first column.
__device__ __forceinline__ void store_rows(const ProductParams& p, int store_bytes,
                                           const uint64_t* acc, bool live, uint32_t* turn,
                                           int64_t slot, int rows, int64_t col, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = live ? pack_bf16x2(__uint_as_float((uint32_t)acc[j * 4 + i]),
                                __uint_as_float((uint32_t)(acc[j * 4 + i] >> 32)))
                  : 0u;
    *reinterpret_cast<uint4*>(turn + lane * 20 + j * 4) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  uint16_t* out = static_cast<uint16_t*>(p.out);
  if (store_bytes == 2) {
    const int64_t n = col + lane;
    for (int r = 0; r < rows; ++r) {
      const uint32_t w = turn[r * 20 + (lane >> 1)];
      if (n < p.N) out[(slot + r) * p.N + n] = (uint16_t)((lane & 1) ? w >> 16 : w & 0xFFFFu);
    }
  } else {
    const int oct = lane & 3;
    const int64_t n = col + oct * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2);
      const uint4 w = *reinterpret_cast<const uint4*>(turn + r * 20 + oct * 4);
      if (r >= rows || n >= p.N) continue;
      uint16_t* o = out + (slot + r) * p.N + n;
      if (store_bytes == 16) {
        *reinterpret_cast<uint4*>(o) = w;
      } else {
        *reinterpret_cast<uint2*>(o) = make_uint2(w.x, w.y);
        if (n + 4 < p.N) reinterpret_cast<uint2*>(o)[1] = make_uint2(w.z, w.w);
      }
    }
  }
  __syncwarp();
}

// The rows of gathered slots, copied by kF8Gather warps: `mine` takes every
// fourth stage, so that a stage's copies have the whole ring's time to land.
// Eight lanes copy a row's 128 bytes, in the swizzled layout that TMA would
// write: 16-byte column j of row r at j ^ (r & 7).  Lane l knows the rows l, l +
// 32, ...  first: the CTA's first slot of a tile; rows: how many it has.
template <int ROWS>
struct RowCopier {
  static constexpr int kHeld = ROWS / 32;
  int32_t held[kHeld];                     // negative: zeros
  __device__ __forceinline__ void start(const ProductParams& p, int64_t first, int rows,
                                        int lane) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      held[i] = -1;
      if (i * 32 + lane < rows) held[i] = p.rows[first + i * 32 + lane];
      if (held[i] >= p.n_a) held[i] = -1;
    }
  }
  // rows, rounded up to `fill`, are written: the others as zeros
  __device__ __forceinline__ void copy(const ProductParams& p, uint32_t dst, int c, int fill,
                                       int lane) {
    const int col = lane & 7, sub = lane >> 3;
    const bool in_row = (int64_t)c * kTcRowBytes + col * 16 < p.H;
    const char* from = static_cast<const char*>(p.a) + col * 16 + (int64_t)c * kTcRowBytes;
    const uint64_t pitch = (uint64_t)p.H;
    dst += sub * kTcRowBytes;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {       // rows i * 32 + j * 4 + sub
        if (i * 32 + j * 4 >= fill) break;
        const int32_t row = __shfl_sync(0xFFFFFFFFu, held[i], j * 4 + sub);
        const bool have = in_row && row >= 0;
        tc::copy16(dst + (i * 32 + j * 4) * kTcRowBytes + ((col ^ ((j * 4 + sub) & 7)) << 4),
                   have ? from + (uint32_t)row * pitch : p.a, have ? 16u : 0u);
      }
    cp_async_commit();
    cp_async_wait<0>();
    tc::fence_async_shared();
  }
};

// What both kernels set up: barriers, tensor memory, groups.
struct Fp8Shared {
  uint32_t base, full, empty, afull, aempty, sfull, sempty;
  Fp8Barriers* bb;
};
__device__ __forceinline__ Fp8Shared fp8_shared(unsigned char* raw, const Fp8Params& t,
                                                unsigned char** smem) {
  Fp8Shared r;
  r.base = (tc::smem_addr(raw) + 1023u) & ~1023u;
  *smem = raw + (r.base - tc::smem_addr(raw));
  r.bb = reinterpret_cast<Fp8Barriers*>(*smem + t.barriers_at);
  r.full = tc::smem_addr(&r.bb->full[0]);
  r.empty = tc::smem_addr(&r.bb->empty[0]);
  r.afull = tc::smem_addr(&r.bb->acc_full[0]);
  r.aempty = tc::smem_addr(&r.bb->acc_empty[0]);
  r.sfull = tc::smem_addr(&r.bb->scale_full[0]);
  r.sempty = tc::smem_addr(&r.bb->scale_empty[0]);
  return r;
}

// After an abort: the stages in flight land before the CTA leaves.
__device__ __forceinline__ void drain_stages(uint32_t full, uint32_t armed, uint32_t NS) {
  for (uint32_t k = armed > NS ? armed - NS : 0; k < armed; ++k) {
    const uint64_t begin = globaltimer_ns();
    while (!tc::mbar_wait_some<true>(full + 8 * (k % NS), (k / NS) & 1, kTcSleepNs) &&
           globaltimer_ns() - begin < kWaitLimitNs) {}
  }
}

// ------------------------------------------------------- a pair of CTAs
// CTA r of a pair has the tile's slots r * 128 .. + 127 (the lanes of its tensor
// memory) and brings, of each half of the weights, the rows r * 64 .. + 63.
//
// Gathered rows have been copied one after the other before (see
// fp8_gather_kernel); p.rows then only says which of the slots have a row.
__global__ void __launch_bounds__(Fp8Pair::kWarps * 32, 1)
farn_fp8_pair_kernel(const __grid_constant__ Fp8Params t,
                     const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_x) {
  using Sh = Fp8Pair;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const ProductParams& p = t.p;
  unsigned char* smem;
  const Fp8Shared m = fp8_shared(smem_raw, t, &smem);
  const uint32_t NS = t.stages;
  const Groups g = groups_at(smem + t.groups_at, p.E);
  volatile int* abort_flag = &m.bb->abort_flag;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // uniform
  const uint32_t rank = cluster_ctarank();

  if (warp == 0) {        // a lane per barrier
    if (lane < (int)NS) {
      mbar_init(m.full + 8 * lane, 1);
      mbar_init(m.empty + 8 * lane, 2);                     // both halves' products
    }
    if (lane < 4) {
      mbar_init(m.afull + 8 * lane, 1);
      mbar_init(m.aempty + 8 * lane, 4 * 2);                // a half's adding warps, both CTAs
    }
    if (lane < kF8ScaleSlots) {
      mbar_init(m.sfull + 8 * lane, 1);
      mbar_init(m.sempty + 8 * lane, kF8Adders);
    }
    if (lane == 0) {
      mbar_init(tc::smem_addr(&m.bb->never), 2);
      m.bb->abort_flag = 0;
    }
    tc::mbar_init_fence();
  }
  if (warp == 9) tc::tmem_alloc<2>(tc::smem_addr(&m.bb->tmem), Sh::kCols);
  if (tid == 8 * 32) {
    tc::prefetch_map(&map_w);
    tc::prefetch_map(&map_x);
  }
  // What does not depend on the kernel before comes before the wait for it: the
  // groups too, unless they are in memory (it took a microsecond behind the wait).
  if (!p.offsets) load_groups(g, p, Sh::kBn);
  tc::fence_before();
  tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = uniform(m.bb->tmem);
  pdl_wait();
  pdl_trigger();
  if (p.offsets) load_groups(g, p, Sh::kBn);       // ends with a block barrier
  const int wts = (int)((p.N + Sh::kTileWeights - 1) / Sh::kTileWeights);
  const int32_t tiles = g.tile[p.E] * wts;
  const int32_t t0 = blockIdx.x / 2, tstep = gridDim.x / 2;
  const int nc = (int)t.HB;
  const int w_rank = (int)rank;
  // slots of a tile that this CTA has
  auto own_slots = [&](const Tile& w) { return min(max(w.n - w_rank * 128, 0), 128); };
  // whether a half of a tile's weights exists
  auto has_half = [&](const Tile& w, int h) {
    return (int64_t)w.wt * Sh::kTileWeights + h * Sh::kHalf < p.N;
  };

  if (warp < kF8Adders)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(Sh::kAddRegs));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(Sh::kRestRegs));

  if (warp < kF8Adders) {
    // ------------------------------------------------- adding and storing
    const int quarter = warp & 3, half = warp >> 2;
    uint32_t sums = tmem + half * Sh::kHalf + ((uint32_t)quarter << 21);
    uint32_t* turn = reinterpret_cast<uint32_t*>(smem + t.part_at) + warp * 32 * 20;
    const uint32_t aempty0 = tc::map_rank(m.aempty, 0);
    const float4* factors = reinterpret_cast<const float4*>(smem + t.scales_at) +
                            half * 128 + quarter * 32 + lane;
    uint32_t ng = 0;                      // groups of factors so far
    // of the next block's buffer: its barriers' offset and phase (the sums' address
    // changes with them: the whole tensor memory is this kernel's)
    uint32_t at = half * 8, phase = 0;
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
      uint64_t acc[Sh::kHalf / 2];
#pragma unroll
      for (int i = 0; i < Sh::kHalf / 2; ++i) acc[i] = 0ull;
      const bool used = has_half(w, half);
      uint32_t v[2][32];
      if (used) {
        ok = f8_wait<kTensor>(m.afull + at, phase, abort_flag, p.err, kErrTcTile);
        if (!ok) break;
        tc::fence_after();
        tc::tmem_ld32(sums, v[0]);
      }
      for (int c0 = 0; ok && c0 < nc; c0 += kF8ScaleBlocks, ++ng) {
        const uint32_t slot = ng % kF8ScaleSlots;
        ok = f8_wait<kOwn>(m.sfull + 8 * slot, ng / kF8ScaleSlots & 1, abort_flag, p.err,
                           kErrTcFull);
        if (!ok) break;
        const float4 f = factors[slot * (Sh::kScaleSlot / 16)];
        __syncwarp();
        arrive_local(m.sempty + 8 * slot, lane);
        if (!used) continue;
#pragma unroll
        for (int j = 0; j < kF8ScaleBlocks; ++j) {
          if (c0 + j >= nc) break;
          const uint64_t s = twice(j == 0 ? f.x : j == 1 ? f.y : j == 2 ? f.z : f.w);
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            tc::tmem_ld_wait();
            tc::tmem_ld32(sums + (q + 1) * 32, v[(q + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              fma_pair(acc[q * 16 + i], v[q & 1][2 * i], v[q & 1][2 * i + 1], s);
          }
          tc::tmem_ld_wait();
          tc::fence_before();       // orders the reads of tensor memory before the arrival
          __syncwarp();
          arrive_relaxed(aempty0 + at, lane);
          // to the next block's buffer
          at ^= 16;
          sums ^= Sh::kTileWeights;
          phase ^= (at >> 4 & 1) ^ 1;
          // its first sums are on their way while the last of this one are added
          const bool more = c0 + j + 1 < nc;
          uint32_t looked = 1;
          if (more) looked = f8_look<kTensor>(m.afull + at, phase);
#pragma unroll
          for (int i = 0; i < 8; ++i) fma_pair(acc[48 + i], v[1][2 * i], v[1][2 * i + 1], s);
          if (more) {
            ok = f8_answer<kTensor>(looked, m.afull + at, phase, abort_flag, p.err, kErrTcTile);
            if (!ok) break;
            tc::fence_after();
            tc::tmem_ld32(sums, v[0]);
          }
#pragma unroll
          for (int i = 8; i < 16; ++i) fma_pair(acc[48 + i], v[1][2 * i], v[1][2 * i + 1], s);
        }
      }
      if (!ok) break;
      const int rows = min(own_slots(w) - quarter * 32, 32);      // of the warp
      if (used && rows > 0) {
        const int64_t slot = (int64_t)w.slot0 + w_rank * 128 + quarter * 32;
        const int64_t n0 = (int64_t)w.wt * Sh::kTileWeights + half * Sh::kHalf;
        bool live = true;
        if (p.rows) {
          const int r = lane < rows ? p.rows[slot + lane] : -1;
          live = r >= 0 && r < t.n_rows;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          store_rows(p, t.store_bytes, acc + q * 16, live, turn, slot, rows, n0 + q * 32, lane);
      }
    }
  } else if (warp == 8) {
    // ---------------------------------- the weights and the slots' rows by TMA
    const uint32_t bar0 = tc::map_rank(m.full, 0);
    RingPos at;
    uint32_t armed = 0;        // stages given to TMA, all but the last NS done
    bool ok = true;
    if (p.stall_test && blockIdx.x == 0)
      ok = tc_wait_warp<false>(tc::smem_addr(&m.bb->never), 0, abort_flag, p.err, kErrTcEmpty);
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
      const bool both = has_half(w, 1);
      const int rows = own_slots(w);
      // both CTAs' boxes; slots come in boxes of 32
      const uint32_t bytes = (both ? 2 : 1) * Sh::kHalf * kTcRowBytes +
                             (w.n + kF8Box - 1) / kF8Box * kF8Box * kTcRowBytes;
      const int n0 = w.wt * Sh::kTileWeights + w_rank * 64;
      for (int c = 0; c < nc; ++c, at.next(NS), ++armed) {
        const uint32_t s = at.stage;
        ok = f8_wait<kCluster>(m.empty + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        const uint32_t to = m.base + s * Sh::kStageBytes;
        if (tc::elect_one()) {
          if (w_rank == 0) mbar_arrive_expect_tx(m.full + 8 * s, bytes);
          tc::load_3d<2>(to + Sh::kSlotBytes, &map_w, c * kTcRowBytes, n0, w.e, bar0 + 8 * s);
          if (both)
            tc::load_3d<2>(to + Sh::kSlotBytes + 64 * kTcRowBytes, &map_w, c * kTcRowBytes,
                           n0 + Sh::kHalf, w.e, bar0 + 8 * s);
#pragma unroll
          for (int i = 0; i < 128 / kF8Box; ++i)
            if (i * kF8Box < rows)
              tc::load_2d<2>(to + i * kF8Box * kTcRowBytes, &map_x, c * kTcRowBytes,
                             w.slot0 + w_rank * 128 + i * kF8Box, bar0 + 8 * s);
        }
        __syncwarp();
      }
    }
    if (*abort_flag && w_rank == 0) drain_stages(m.full, armed, NS);
  } else if (warp == 9 || warp == 10) {
    // ---------------------- matrix instructions: a warp for each half's weights
    // (one warp's waits and issues for both took 650 cycles a block, more than
    // the products' 512)
    if (w_rank == 0) {
      const int h = warp - 9;
      RingPos at;
      uint32_t nb = 0;                     // blocks of this half so far
      bool ok = true;
      const uint64_t desc0 = tc::operand_desc(m.base);
      const uint32_t idesc = tc::idesc_e4m3(256, Sh::kHalf);
      for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
        const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
        const bool used = has_half(w, h);
        for (int c = 0; c < nc; ++c, at.next(NS)) {
          const uint32_t s = at.stage;
          ok = f8_wait<kCluster>(m.full + 8 * s, at.phase, abort_flag, p.err, kErrTcFull);
          if (!ok) break;
          if (used) {
            const uint32_t b = nb & 1, bar = (b * 2 + h) * 8;
            ok = f8_wait<kTensor>(m.aempty + bar, ((nb >> 1) & 1) ^ 1, abort_flag, p.err,
                                  kErrTcTile);
            if (!ok) break;
            tc::fence_after();
            const uint64_t da = desc0 + (s * Sh::kStageBytes >> 4);
            const uint64_t db = da + ((Sh::kSlotBytes + h * 64 * kTcRowBytes) >> 4);
            const uint32_t d = tmem + b * Sh::kTileWeights + h * Sh::kHalf;
            if (tc::elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc::mma_fp8<2>(d, da + 2 * k, db + 2 * k, idesc, k > 0 ? 1u : 0u);
              tc::commit<2>(m.afull + bar);
              tc::commit<2>(m.empty + 8 * s);
            }
            ++nb;
          } else if (tc::elect_one()) {
            tc::commit<2>(m.empty + 8 * s);
          }
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- factors
    // sa * sb of the CTA's 128 slots and both blocks of weights, for four blocks
    // of the row at a time: lane l has the slots l, l + 32, ...
    float4* to0 = reinterpret_cast<float4*>(smem + t.scales_at) + lane;
    const bool vec = t.scale_vec;
    uint32_t ng = 0;
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
      const float *ra[4], *rb[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ra[i] = nullptr;
        if (i * 32 + lane < own_slots(w)) {
          const int64_t r = (int64_t)w.slot0 + w_rank * 128 + i * 32 + lane;
          if (r < p.n_a) ra[i] = t.a_scale + r * t.HB;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t wb = (int64_t)w.wt * 2 + h;
        rb[h] = wb < t.NB ? t.b_scale + ((int64_t)w.e * t.NB + wb) * t.HB : nullptr;
      }
      for (int c = 0; c < nc; c += kF8ScaleBlocks, ++ng) {
        const uint32_t slot = ng % kF8ScaleSlots;
        ok = f8_wait<kOwn>(m.sempty + 8 * slot, (ng / kF8ScaleSlots & 1) ^ 1, abort_flag, p.err,
                     kErrTcEmpty);
        if (!ok) break;
        float4* to = to0 + slot * (Sh::kScaleSlot / 16);
        float4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = load_scales(ra[i], c, nc, vec);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 b = load_scales(rb[h], c, nc, vec);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            to[h * 128 + i * 32] =
                make_float4(a[i].x * b.x, a[i].y * b.y, a[i].z * b.z, a[i].w * b.w);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(m.sfull + 8 * slot);
      }
    }
  }

  // As in farn_product_tc_kernel: after an abort the tensor cores may still be
  // at work on what they were given.
  __syncthreads();
  if (*abort_flag && (warp == 9 || warp == 10) && w_rank == 0) {
    const uint32_t never = tc::smem_addr(&m.bb->never);      // both warps' commits
    if (tc::elect_one()) tc::commit<2>(never);
    __syncwarp();
    const uint64_t begin = globaltimer_ns();
    while (!tc::mbar_wait_some<true>(never, 0, kTcSleepNs) &&
           globaltimer_ns() - begin < kWaitLimitNs) {}
  }
  tc::fence_before();
  tc::cluster_sync();
  tc::fence_after();
  if (warp == 9) tc::tmem_free<2>(tmem, Sh::kCols);
}

// ------------------------------------------------------- rows side by side
// The rows of a long call's slots and their scales, copied to where `pair`
// reads them with TMA: every row is read once here instead of once for every 256
// weights there.  (4096 tokens of 8 experts, 7168 -> 4096: 912 us, 844 of them the
// product; with the rows copied by the tile's own warps 1557, fetched by TMA four
// rows to an instruction from the tile's own order 2360.)  A slot without a row gets
// zeros.  16 bytes of a row per thread and step; a warp per slot.
struct Fp8GatherParams {
  const uint8_t* x;
  const float* x_scale;
  const int32_t* rows;
  uint8_t* to;
  float* to_scale;
  int64_t n_rows, S, H, HB;
};
constexpr int kF8CopyThreads = 256;

__global__ void __launch_bounds__(kF8CopyThreads)
fp8_gather_kernel(const Fp8GatherParams g) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t s = (int64_t)blockIdx.x * (kF8CopyThreads / 32) + (threadIdx.x >> 5);
  if (s >= g.S) return;
  const int64_t r = g.rows[s];
  const bool live = r >= 0 && r < g.n_rows;
  const uint4* from = reinterpret_cast<const uint4*>(g.x + (live ? r : 0) * g.H);
  uint4* to = reinterpret_cast<uint4*>(g.to + s * g.H);
  const int64_t n = g.H / 16;
  for (int64_t i = lane; i < n; i += 128) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (live && i + j * 32 < n) v[j] = __ldg(from + i + j * 32);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j * 32 < n) to[i + j * 32] = v[j];
  }
  for (int64_t i = lane; i < g.HB; i += 32)
    g.to_scale[s * g.HB + i] = live ? __ldg(g.x_scale + r * g.HB + i) : 0.0f;
}

// --------------------------------------------------------------- one CTA
template <bool GATHER>
__global__ void __launch_bounds__(Fp8One<GATHER>::kWarps * 32, 1)
farn_fp8_one_kernel(const __grid_constant__ Fp8Params t,
                    const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_x) {
  using Sh = Fp8One<GATHER>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const ProductParams& p = t.p;
  unsigned char* smem;
  const Fp8Shared m = fp8_shared(smem_raw, t, &smem);
  const uint32_t NS = t.stages;
  const Groups g = groups_at(smem + t.groups_at, p.E);
  volatile int* abort_flag = &m.bb->abort_flag;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // uniform
  const uint32_t rank = cluster_ctarank();
  const int csize = t.ks;

  if (warp == 0) {        // a lane per barrier
    if (lane < (int)NS) {
      mbar_init(m.full + 8 * lane, GATHER ? 2 : 1);         // TMA; gathered rows
      mbar_init(m.empty + 8 * lane, 1);
    }
    if (lane < Sh::kBufs) {
      mbar_init(m.afull + 8 * lane, 1);
      mbar_init(m.aempty + 8 * lane, kF8Adders);
    }
    if (lane < kF8ScaleSlots) {
      mbar_init(m.sfull + 8 * lane, 1);
      mbar_init(m.sempty + 8 * lane, kF8Adders);
    }
    if (lane == 0) {
      mbar_init(tc::smem_addr(&m.bb->part_full), kF8Adders * csize);
      mbar_init(tc::smem_addr(&m.bb->part_empty), kF8Adders * csize);
      mbar_init(tc::smem_addr(&m.bb->never), 1);
      m.bb->abort_flag = 0;
    }
    tc::mbar_init_fence();
  }
  if (warp == 9) tc::tmem_alloc<1>(tc::smem_addr(&m.bb->tmem), Sh::kCols);
  if (tid == 8 * 32) {
    tc::prefetch_map(&map_w);
    if constexpr (!GATHER) tc::prefetch_map(&map_x);
  }
  if (!p.offsets) load_groups(g, p, Sh::kBn);      // as in the pair
  tc::fence_before();
  if (csize > 1) tc::cluster_sync(); else __syncthreads();
  tc::fence_after();
  const uint32_t tmem = uniform(m.bb->tmem);
  pdl_wait();
  pdl_trigger();
  if (p.offsets) load_groups(g, p, Sh::kBn);

  const int wts = (int)((p.N + Sh::kTileWeights - 1) / Sh::kTileWeights);
  const int32_t tiles = g.tile[p.E] * wts;
  const int32_t t0 = blockIdx.x / csize, tstep = gridDim.x / csize;
  const int chunks = (int)t.HB;
  const int c0 = (int)((int64_t)chunks * rank / csize);
  const int c1 = (int)((int64_t)chunks * (rank + 1) / csize);
  const int nc = c1 - c0;
  auto filled = [&](const Tile& w) { return (w.n + 15) / 16 * 16; };   // the N side

  if (warp < kF8Adders) {
    // ------------------------------------------------- adding and storing
    const int quarter = warp & 3;
    const int cols0 = (warp >> 2) * Sh::kWarpCols;            // the warp's first column
    const uint32_t sums = tmem + cols0 + ((uint32_t)quarter << 21);
    const float* scales = reinterpret_cast<const float*>(smem + t.scales_at) + cols0;
    uint32_t* turn = reinterpret_cast<uint32_t*>(smem + t.part_at + warp * kTurnBytes);
    float* part = reinterpret_cast<float*>(smem + t.part_at);
    const uint32_t part_full = tc::smem_addr(&m.bb->part_full);
    const uint32_t part_empty = tc::smem_addr(&m.bb->part_empty);
    uint32_t ng = 0, nt = 0;               // groups of scales, tiles so far
    uint32_t buf = 0, phase = 0;           // the next block's sums
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep, ++nt) {
      const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
      const int mine = min(max(w.n - cols0, 0), Sh::kWarpCols);   // columns in use
      float acc[Sh::kWarpCols];
#pragma unroll
      for (int i = 0; i < Sh::kWarpCols; ++i) acc[i] = 0.0f;
      uint32_t looked = f8_look<kOwn>(m.afull + 8 * buf, phase);
      for (int c = 0; ok && c < nc; ++ng) {
        const uint32_t slot = ng % kF8ScaleSlots;
        ok = f8_wait<kOwn>(m.sfull + 8 * slot, ng / kF8ScaleSlots & 1, abort_flag, p.err,
                           kErrTcFull);
        if (!ok) break;
        const int end = min(nc, c + kF8ScaleBlocks);
        const float* s = scales + slot * (Sh::kScaleSlot / 4);
        for (; c < end; ++c, s += Sh::kBn) {
          ok = f8_answer<kOwn>(looked, m.afull + 8 * buf, phase, abort_flag, p.err, kErrTcTile);
          if (!ok) break;
          tc::fence_after();
          const uint32_t d = sums + buf * Sh::kBn, bar = m.aempty + 8 * buf;
          uint32_t v[2][16];
#pragma unroll
          for (int q = 0; q < Sh::kWarpCols / 16; ++q)
            if (q * 16 < mine) tc::tmem_ld16(d + q * 16, v[q]);
          if (++buf == Sh::kBufs) { buf = 0; phase ^= 1; }
          if (c + 1 < nc) looked = f8_look<kOwn>(m.afull + 8 * buf, phase);
          tc::tmem_ld_wait();
          tc::fence_before();       // orders the reads of tensor memory before the arrival
          __syncwarp();
          arrive_local(bar, lane);
#pragma unroll
          for (int q = 0; q < Sh::kWarpCols / 16; ++q) {
            if (q * 16 < mine) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float4 sv = *reinterpret_cast<const float4*>(s + q * 16 + j * 4);
                float* to = acc + q * 16 + j * 4;
                to[0] = fmaf(__uint_as_float(v[q][4 * j]), sv.x, to[0]);
                to[1] = fmaf(__uint_as_float(v[q][4 * j + 1]), sv.y, to[1]);
                to[2] = fmaf(__uint_as_float(v[q][4 * j + 2]), sv.z, to[2]);
                to[3] = fmaf(__uint_as_float(v[q][4 * j + 3]), sv.w, to[3]);
              }
            }
          }
        }
        __syncwarp();
        if (ok) arrive_local(m.sempty + 8 * slot, lane);
      }
      if (!ok) break;
      const int64_t n0 = (int64_t)w.wt * Sh::kTileWeights;
      if (csize == 1) {
        if (mine > 0) {
          const int64_t slot = (int64_t)w.slot0 + cols0;
          uint32_t live = 0xFFFFFFFFu;
          if constexpr (GATHER) {
            const int r = lane < mine ? p.rows[slot + lane] : -1;
            live = __ballot_sync(0xFFFFFFFFu, r >= 0 && r < p.n_a);
          }
          uint32_t v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(acc[j]);
          store_columns<GATHER>(p, t.store_bytes, v, turn, slot, mine, live, n0 + quarter * 32,
                                lane);
        }
      } else {
        // the other CTAs have read this one's last part
        ok = tc_wait_warp<true>(part_empty, (nt & 1) ^ 1, abort_flag, p.err, kErrTcJoin);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < Sh::kWarpCols; ++i)
          if (i < mine) part[(cols0 + i) * kPartPitch + quarter * 32 + lane] = acc[i];
        __syncwarp();
        if (lane < csize) tc::mbar_arrive_cluster(tc::map_rank(part_full, lane));
        ok = tc_wait_warp<true>(part_full, nt & 1, abort_flag, p.err, kErrTcJoin);
        if (!ok) break;
        // each CTA sums its share of the tile, four weights to a thread, the
        // parts in rank order.  (Parts written to the CTA that sums them, rather
        // than read by it, took longer: 1 x 4096 x 4096 8.3 us, 7.9 this way.)
        const uint32_t from = tc::smem_addr(part);
        const int quads = w.n * (kTcWeights / 4);
        uint16_t* out = static_cast<uint16_t*>(p.out);
        for (int i = (int)rank * kF8Adders * 32 + tid; i < quads; i += csize * kF8Adders * 32) {
          const uint32_t at = ((i >> 5) * kPartPitch + (i & 31) * 4) * 4;
          float4 v[kTcMaxSplit];
#pragma unroll
          for (int q = 0; q < kTcMaxSplit; ++q)
            if (q < csize) v[q] = tc::ld_cluster_v4(tc::map_rank(from, q) + at);
          float4 sum = v[0];
#pragma unroll
          for (int q = 1; q < kTcMaxSplit; ++q)
            if (q < csize) {
              sum.x += v[q].x; sum.y += v[q].y; sum.z += v[q].z; sum.w += v[q].w;
            }
          const int64_t s = (int64_t)w.slot0 + (i >> 5), n = n0 + (i & 31) * 4;
          if constexpr (GATHER)
            if (p.rows[s] < 0 || p.rows[s] >= p.n_a) sum = make_float4(0.f, 0.f, 0.f, 0.f);
          const uint32_t e[2] = {pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w)};
          uint16_t* o = out + s * p.N + n;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (t.store_bytes >= 8) {
              if (n + 2 * k < p.N) reinterpret_cast<uint32_t*>(o)[k] = e[k];
            } else {
              if (n + 2 * k < p.N) o[2 * k] = (uint16_t)(e[k] & 0xFFFFu);
              if (n + 2 * k + 1 < p.N) o[2 * k + 1] = (uint16_t)(e[k] >> 16);
            }
          }
        }
        __syncwarp();
        if (lane < csize) tc::mbar_arrive_cluster(tc::map_rank(part_empty, lane));
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------- weights' producer
    const uint32_t bar0 = tc::map_rank(m.full, rank);
    RingPos at;
    uint32_t armed = 0;        // stages given to TMA, all but the last NS done
    bool ok = true;
    if (p.stall_test && blockIdx.x == 0)
      ok = tc_wait_warp<false>(tc::smem_addr(&m.bb->never), 0, abort_flag, p.err, kErrTcEmpty);
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
      const uint32_t bytes =
          Sh::kABytes + (GATHER ? 0 : (filled(w) + kF8Box - 1) / kF8Box * kF8Box * kTcRowBytes);
      for (int c = c0; c < c1; ++c, at.next(NS), ++armed) {
        const uint32_t s = at.stage;
        ok = f8_wait<kOwn>(m.empty + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        if (tc::elect_one()) {
          mbar_arrive_expect_tx(m.full + 8 * s, bytes);
          tc::load_3d<1>(m.base + s * Sh::kStageBytes, &map_w, c * kTcRowBytes,
                         w.wt * Sh::kTileWeights, w.e, bar0 + 8 * s);
          tc::load_3d<1>(m.base + s * Sh::kStageBytes + 64 * kTcRowBytes, &map_w, c * kTcRowBytes,
                         w.wt * Sh::kTileWeights + 64, w.e, bar0 + 8 * s);
        }
        __syncwarp();
      }
    }
    if (*abort_flag) drain_stages(m.full, armed, NS);
  } else if (warp == 9) {
    // ------------------------------------------------- matrix instructions
    RingPos at;
    uint32_t buf = 0, phase = 0;           // the next block's sums
    bool ok = true;
    const uint64_t desc0 = tc::operand_desc(m.base);
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
      const uint32_t idesc = tc::idesc_e4m3(kTcWeights, filled(w));
      for (int c = 0; c < nc; ++c, at.next(NS)) {
        const uint32_t s = at.stage;
        const uint32_t free = f8_look<kOwn>(m.aempty + 8 * buf, phase ^ 1);
        ok = f8_wait<kOwn>(m.full + 8 * s, at.phase, abort_flag, p.err, kErrTcFull) &&
             f8_answer<kOwn>(free, m.aempty + 8 * buf, phase ^ 1, abort_flag, p.err, kErrTcTile);
        if (!ok) break;
        tc::fence_after();
        const uint64_t da = desc0 + (s * Sh::kStageBytes >> 4), db = da + (Sh::kABytes >> 4);
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_fp8<1>(tmem + buf * Sh::kBn, da + 2 * k, db + 2 * k, idesc, k > 0 ? 1u : 0u);
          tc::commit<1>(m.afull + 8 * buf);
          tc::commit<1>(m.empty + 8 * s);
        }
        if (++buf == Sh::kBufs) { buf = 0; phase ^= 1; }
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // -------------------------------------------------------------- scales
    // Lane l has the slots l and l + 32: sa * sb, a block's slots one after the
    // other.
    float* to0 = reinterpret_cast<float*>(smem + t.scales_at) + lane;
    const bool vec = t.scale_vec;
    uint32_t ng = 0;
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
      const float* row[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int s = i * 32 + lane;
        row[i] = nullptr;
        if (s < w.n) {
          int64_t r = (int64_t)w.slot0 + s;
          if constexpr (GATHER) r = p.rows[r];
          if (r >= 0 && r < p.n_a) row[i] = t.a_scale + r * t.HB;
        }
      }
      const float* sb = t.b_scale + ((int64_t)w.e * t.NB + w.wt) * t.HB;
      for (int c = c0; c < c1; c += kF8ScaleBlocks, ++ng) {
        const float4 vb = load_scales(sb, c, c1, vec);
        const float4 v[2] = {load_scales(row[0], c, c1, vec), load_scales(row[1], c, c1, vec)};
        const uint32_t slot = ng % kF8ScaleSlots;
        ok = f8_wait<kOwn>(m.sempty + 8 * slot, (ng / kF8ScaleSlots & 1) ^ 1, abort_flag,
                                 p.err, kErrTcEmpty);
        if (!ok) break;
        float* to = to0 + slot * (Sh::kScaleSlot / 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          to[i * 32] = v[i].x * vb.x;
          to[Sh::kBn + i * 32] = v[i].y * vb.y;
          to[2 * Sh::kBn + i * 32] = v[i].z * vb.z;
          to[3 * Sh::kBn + i * 32] = v[i].w * vb.w;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(m.sfull + 8 * slot);
      }
    }
  } else if (!GATHER && warp == 10) {
    // --------------------------------------------------- slots' producer
    const uint32_t bar0 = tc::map_rank(m.full, rank);
    RingPos at;
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
      for (int c = c0; c < c1; ++c, at.next(NS)) {
        const uint32_t s = at.stage;
        ok = f8_wait<kOwn>(m.empty + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        if (tc::elect_one()) {
#pragma unroll
          for (int i = 0; i < Sh::kBn / kF8Box; ++i)
            if (i * kF8Box < filled(w))
              tc::load_2d<1>(m.base + s * Sh::kStageBytes + Sh::kABytes + i * kF8Box * kTcRowBytes,
                             &map_x, c * kTcRowBytes, w.slot0 + i * kF8Box, bar0 + 8 * s);
        }
        __syncwarp();
      }
    }
  } else if (GATHER && (warp == 10 || warp >= 12) && warp < 12 + kF8Gather - 1) {
    // -------------------------------------------------------- gathered rows
    const int mine = warp == 10 ? 0 : warp - 11;
    RowCopier<64> rows;
    RingPos at;
    at.skip(mine, NS);
    int ahead = mine;
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, Sh::kBn);
      rows.start(p, w.slot0, w.n, lane);
      int c = c0 + ahead;
      for (; c < c1; c += kF8Gather, at.skip(kF8Gather, NS)) {
        const uint32_t s = at.stage;
        ok = f8_wait<kOwn>(m.empty + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        rows.copy(p, m.base + s * Sh::kStageBytes + Sh::kABytes, c, filled(w), lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(m.full + 8 * s);
      }
      ahead = c - c1;
    }
  }

  // As in farn_product_tc_kernel: after an abort the tensor cores may still be
  // at work on what they were given.
  __syncthreads();
  if (*abort_flag && warp == 9) {
    const uint32_t never = tc::smem_addr(&m.bb->never);
    if (tc::elect_one()) tc::commit<1>(never);
    __syncwarp();
    const uint64_t begin = globaltimer_ns();
    while (!tc::mbar_wait_some<true>(never, 0, kTcSleepNs) &&
           globaltimer_ns() - begin < kWaitLimitNs) {}
  }
  tc::fence_before();
  if (csize > 1) tc::cluster_sync(); else __syncthreads();
  tc::fence_after();
  if (warp == 9) tc::tmem_free<1>(tmem, Sh::kCols);
}

// ------------------------------------------------------------ any shape
// As farn_product_plain_kernel, with a block's sum scaled when it is complete.
__global__ void __launch_bounds__(kPlainThreads)
farn_fp8_product_plain_kernel(const Fp8Params t) {
  const ProductParams& p = t.p;
  __shared__ int32_t gmem[groups_bytes(kMaxExperts) / 4];
  const Groups g = groups_at(gmem, p.E);
  __shared__ float as[kPlainK][kPlainTile + 1], bs[kPlainK][kPlainTile + 1];
  pdl_wait();
  pdl_trigger();
  load_groups(g, p, kPlainTile);
  const int tid = threadIdx.x, ti = tid / 16, tj = tid % 16;
  const int wts = (int)((p.N + kPlainTile - 1) / kPlainTile);
  const int32_t tiles = g.tile[p.E] * wts;
  for (int32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Tile w = find_tile(g, p.E, tile, wts, kPlainTile);
    const int64_t n0 = (int64_t)w.wt * kPlainTile;
    int64_t row[4];                        // -1: zeros
    for (int i = 0; i < 4; ++i) {
      const int r = ti * 4 + i;
      row[i] = -1;
      if (r < w.n) row[i] = p.rows ? p.rows[w.slot0 + r] : (int64_t)w.slot0 + r;
      if (row[i] >= p.n_a) row[i] = -1;
    }
    // a tile's 64 weights lie in one block of 128
    const float* sb = t.b_scale + ((int64_t)w.e * t.NB + n0 / kFp8Block) * t.HB;
    float acc[4][4] = {}, sum[4][4] = {};
    for (int64_t h0 = 0; h0 < p.H; h0 += kPlainK) {
      for (int i = tid; i < kPlainTile * kPlainK; i += kPlainThreads) {
        const int r = i / kPlainK, k = i % kPlainK;
        const int64_t h = h0 + k;
        float va = 0.0f, vb = 0.0f;
        if (h < p.H && r < w.n) {
          const int64_t at = p.rows ? p.rows[w.slot0 + r] : (int64_t)w.slot0 + r;
          if (at >= 0 && at < p.n_a)
            va = e4m3_to_f32(static_cast<const uint8_t*>(p.a)[at * p.H + h]);
        }
        if (h < p.H && n0 + r < p.N)
          vb = e4m3_to_f32(
              static_cast<const uint8_t*>(p.b)[((int64_t)w.e * p.N + n0 + r) * p.H + h]);
        as[k][r] = va;
        bs[k][r] = vb;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kPlainK; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            sum[i][j] = fmaf(as[k][ti * 4 + i], bs[k][tj + 16 * j], sum[i][j]);
      __syncthreads();
      if ((h0 + kPlainK) % kFp8Block == 0 || h0 + kPlainK >= p.H) {
        const int64_t b = h0 / kFp8Block;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = row[i] >= 0 ? t.a_scale[row[i] * t.HB + b] * sb[b] : 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][j] = fmaf(sum[i][j], s, acc[i][j]);
            sum[i][j] = 0.0f;
          }
        }
      }
    }
    for (int i = 0; i < 4; ++i) {
      const int r = ti * 4 + i;
      if (r >= w.n) break;
      for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + tj + 16 * j;
        if (n < p.N)
          static_cast<uint16_t*>(p.out)[((int64_t)w.slot0 + r) * p.N + n] =
              row[i] >= 0 ? to_bf16(acc[i][j]) : (uint16_t)0;
      }
    }
  }
}

}  // namespace farn

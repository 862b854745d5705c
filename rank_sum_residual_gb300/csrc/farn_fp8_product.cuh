// The FP8 products: E4M3 codes with an fp32 scale for every 128 elements of a
// slot's row and every 128 x 128 of the weights.
//
//     out[s, n] = sum_b (sa[s, b] * sb[n / 128, b]) * sum_{h in b} a[s, h] * b[n, h]
//
// The inner sums are matrix instructions of one block's 128 bytes of a row
// (one stage of the ring); the outer sum is fp32 multiply-adds in registers,
// because the matrix instructions know scales of blocks of 32 with powers of
// two only.  As in the other products the weights are the M side, so a CTA's
// 128 weights share one sb per block, a slot's scale is a column's, and the
// products sa * sb reach the adding warps through shared memory.
//
//   CG = 2  pairs of CTAs share a tile of 256 weights by 256 slots: long calls
//   CG = 1  one CTA per tile of 128 weights by 64 slots; up to four CTAs of a
//           cluster split the row and join their sums, in rank order, through
//           distributed shared memory: short calls
//
// Warps of a CTA: eight that add (a quarter of the weights and half of the
// columns each) and store; one that has TMA fetch the weights, one that issues
// the matrix instructions, one that has TMA fetch the slots' rows, or four that
// copy gathered rows themselves; two that fetch the scales.
//
// The tensor memory holds two blocks' sums, each in halves of 128 columns that
// are handed over by themselves: a half is read while the next three are
// computed, which hides the hand-over (commit, wait, read, arrive).
//
// Every wait is bounded (see tc_wait).
#pragma once

#include <cuda.h>

#include "farn_fp8.cuh"
#include "farn_product_tc.cuh"

namespace farn {

constexpr int kF8Adders = 8;           // warps
constexpr int kF8Warps = 16;
constexpr int kF8Box = 32;             // slots' rows of a TMA box
constexpr int kF8ScaleBlocks = 4;      // blocks of a row whose scales are fetched together
constexpr int kF8ScaleSlots = 3;
constexpr int kF8ScaleWarps = 2;
// Registers: of a thread at launch, and once the adding warps of a pair's tile
// have taken some from the others (half of the warps each).
constexpr int kF8Regs = 128, kF8AddRegs = 200, kF8RestRegs = 56;
static_assert(kF8AddRegs + kF8RestRegs <= 2 * kF8Regs && 2 * kF8Adders == kF8Warps, "");
constexpr int kF8Gather = 4;           // warps; not more than the ring has stages

struct Fp8Params {
  ProductParams p;                     // a, b: E4M3 codes
  const float* a_scale;                // [n_a, HB]
  const float* b_scale;                // [E, NB, HB]
  int64_t HB, NB;
  int scale_vec;                       // a_scale's rows can be read 16 bytes at a time
  int stages;
  int ks;                              // CTAs of a cluster that split the row (CG = 1)
  int store_bytes;                     // see store_columns
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

template <int CG, int BN, bool GATHER>
struct Fp8Shape {
  static constexpr int kHalves = BN > 128 ? 2 : 1;        // parts of a buffer handed over alone
  static constexpr int kHalf = BN / kHalves;              // columns of one
  static constexpr int kWarpCols = BN / 2;                // columns of an adding warp
  static constexpr int kRows = BN / CG;                   // slots' rows per CTA
  static constexpr int kABytes = kTcWeights * kTcRowBytes;
  static constexpr int kBBytes = kRows * kTcRowBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kScaleSlot = kF8ScaleBlocks * BN * 4;
  static constexpr int kCols = 2 * BN < 128 ? 128 : 2 * BN;
  static constexpr int kStep = 16 * CG;                   // granularity of a half's slots
  static constexpr int kLaneSlots = BN / (32 * kF8ScaleWarps);
  static_assert(kHalf / CG % kF8Box == 0 && kWarpCols % 32 == 0, "");
  static_assert(kHalves == 1 || kWarpCols == kHalf, "an adding warp's columns are one half");
};

// d += a * b for two fp32 values each; one rounding per value.
__device__ __forceinline__ void fma2(uint64_t& d, uint32_t a0, uint32_t a1, uint64_t b) {
  asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
      : "+l"(d) : "r"(a0), "r"(a1), "l"(b));
}

// The half h of a tile's slots: how many there are, as the matrix
// instruction's N.
template <typename Sh>
__device__ __forceinline__ int half_slots(const Tile& w, int h) {
  const int n = min(w.n - h * Sh::kHalf, Sh::kHalf);
  return n <= 0 ? 0 : (n + Sh::kStep - 1) / Sh::kStep * Sh::kStep;
}

template <int CG, int BN, bool GATHER>
__global__ void __launch_bounds__(kF8Warps * 32, 1)
farn_fp8_product_kernel(const __grid_constant__ Fp8Params t,
                        const __grid_constant__ CUtensorMap map_w,
                        const __grid_constant__ CUtensorMap map_x) {
  using Sh = Fp8Shape<CG, BN, GATHER>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const ProductParams& p = t.p;
  const uint32_t base = (tc::smem_addr(smem_raw) + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - tc::smem_addr(smem_raw));
  const uint32_t NS = t.stages;
  Fp8Barriers* bb = reinterpret_cast<Fp8Barriers*>(smem + t.barriers_at);
  const Groups g = groups_at(smem + t.groups_at, p.E);
  const uint32_t full0 = tc::smem_addr(&bb->full[0]);
  const uint32_t empty0 = tc::smem_addr(&bb->empty[0]);
  const uint32_t afull0 = tc::smem_addr(&bb->acc_full[0]);
  const uint32_t aempty0 = tc::smem_addr(&bb->acc_empty[0]);
  const uint32_t sfull0 = tc::smem_addr(&bb->scale_full[0]);
  const uint32_t sempty0 = tc::smem_addr(&bb->scale_empty[0]);
  volatile int* abort_flag = &bb->abort_flag;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // uniform
  const uint32_t rank = cluster_ctarank();
  const int csize = CG == 2 ? 2 : t.ks;

  if (warp == 0) {        // a lane per barrier
    if (lane < (int)NS) {
      mbar_init(full0 + 8 * lane, GATHER ? 1 + CG : 1);   // TMA; gathered rows
      mbar_init(empty0 + 8 * lane, 1);
    }
    if (lane < 4) {
      mbar_init(afull0 + 8 * lane, 1);
      mbar_init(aempty0 + 8 * lane, kF8Adders / Sh::kHalves * CG);
    }
    if (lane < kF8ScaleSlots) {
      mbar_init(sfull0 + 8 * lane, kF8ScaleWarps);
      mbar_init(sempty0 + 8 * lane, kF8Adders);
    }
    if (lane == 0) {
      mbar_init(tc::smem_addr(&bb->part_full), kF8Adders * csize);
      mbar_init(tc::smem_addr(&bb->part_empty), kF8Adders * csize);
      mbar_init(tc::smem_addr(&bb->never), 1);
      bb->abort_flag = 0;
    }
    tc::mbar_init_fence();
  }
  if (warp == 9) tc::tmem_alloc<CG>(tc::smem_addr(&bb->tmem), Sh::kCols);
  if (tid == 8 * 32) {
    tc::prefetch_map(&map_w);
    if constexpr (!GATHER) tc::prefetch_map(&map_x);
  }
  pdl_wait();
  pdl_trigger();
  load_groups(g, p, BN);            // ends with a block barrier
  tc::fence_before();
  if (csize > 1) tc::cluster_sync(); else __syncthreads();
  tc::fence_after();
  const uint32_t tmem = uniform(bb->tmem);

  constexpr int kTileWeights = kTcWeights * CG;
  constexpr bool kPair = CG == 2;   // the other CTA arrives on the tile's barriers too
  const int wts = (int)((p.N + kTileWeights - 1) / kTileWeights);
  const int32_t tiles = g.tile[p.E] * wts;
  const int32_t t0 = blockIdx.x / csize, tstep = gridDim.x / csize;
  const int chunks = (int)t.HB;
  const int c0 = CG == 2 ? 0 : (int)((int64_t)chunks * rank / csize);
  const int c1 = CG == 2 ? chunks : (int)((int64_t)chunks * (rank + 1) / csize);
  const int nc = c1 - c0;
  const int w_rank = CG == 2 ? (int)rank : 0;      // this CTA's part of a tile's weights

  // The adding warps of a pair's tile hold 128 sums each.
  if constexpr (Sh::kWarpCols == 128) {
    if (warp < kF8Adders)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kF8AddRegs));
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kF8RestRegs));
  }

  if (warp < kF8Adders) {
    // ------------------------------------------------- adding and storing
    const int quarter = warp & 3, part_of = warp >> 2;
    const int half = Sh::kHalves == 2 ? part_of : 0;
    const uint32_t cols0 = part_of * Sh::kWarpCols;            // the warp's first column
    const uint32_t lanes_at = (uint32_t)quarter << 21;         // its lanes of tensor memory
    const float* scales = reinterpret_cast<const float*>(smem + t.scales_at) + cols0;
    uint32_t* turn = reinterpret_cast<uint32_t*>(smem + t.part_at + warp * kTurnBytes);
    float* part = reinterpret_cast<float*>(smem + t.part_at);
    const uint32_t part_full = tc::smem_addr(&bb->part_full);
    const uint32_t part_empty = tc::smem_addr(&bb->part_empty);
    uint32_t nb = 0, ng = 0, nt = 0;       // blocks of this half, groups of scales, tiles so far
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep, ++nt) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      const int mine = min(max(w.n - (int)cols0, 0), Sh::kWarpCols);   // columns in use
      const bool used = Sh::kHalves == 1 || mine > 0;
      uint64_t acc[Sh::kWarpCols / 2];
#pragma unroll
      for (int i = 0; i < Sh::kWarpCols / 2; ++i) acc[i] = 0ull;
      for (int c = 0; ok && c < nc; ++ng) {
        const uint32_t slot = ng % kF8ScaleSlots;
        ok = tc_wait_warp<false>(sfull0 + 8 * slot, ng / kF8ScaleSlots & 1, abort_flag, p.err,
                                 kErrTcFull);
        if (!ok) break;
        const int end = min(nc, c + kF8ScaleBlocks);
        const float* s = scales + slot * (Sh::kScaleSlot / 4);
        if (used) {
          for (; c < end; ++c, ++nb, s += BN) {
            const uint32_t b = nb & 1, at = (b * 2 + half) * 8;
            ok = tc_wait_warp<kPair>(afull0 + at, (nb >> 1) & 1, abort_flag, p.err, kErrTcTile);
            if (!ok) break;
            tc::fence_after();
            const uint32_t d = tmem + b * BN + cols0 + lanes_at;
#pragma unroll
            for (int q = 0; q < Sh::kWarpCols / 32; ++q) {
              if (q * 32 < mine) {
                uint32_t v[32];
                tc::tmem_ld32(d + q * 32, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const ulonglong2 sv = *reinterpret_cast<const ulonglong2*>(s + q * 32 + j * 4);
                  fma2(acc[q * 16 + j * 2], v[4 * j], v[4 * j + 1], sv.x);
                  fma2(acc[q * 16 + j * 2 + 1], v[4 * j + 2], v[4 * j + 3], sv.y);
                }
              }
            }
            tc::fence_before();       // orders the reads of tensor memory before the arrival
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_first<CG>(aempty0 + at);
          }
        } else {
          c = end;
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(sempty0 + 8 * slot);
      }
      if (!ok) break;
      const int64_t n0 = (int64_t)w.wt * kTileWeights + w_rank * kTcWeights;
      const bool split = CG == 1 && csize > 1;
      if (!split) {
#pragma unroll
        for (int q = 0; q < Sh::kWarpCols / 32; ++q) {
          if (q * 32 < mine) {
            const int64_t slot = (int64_t)w.slot0 + cols0 + q * 32;
            uint32_t live = 0xFFFFFFFFu;
            if constexpr (GATHER) {
              const int r = q * 32 + lane < mine ? p.rows[slot + lane] : -1;
              live = __ballot_sync(0xFFFFFFFFu, r >= 0 && r < p.n_a);
            }
            uint32_t v[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              v[2 * j] = (uint32_t)acc[q * 16 + j];
              v[2 * j + 1] = (uint32_t)(acc[q * 16 + j] >> 32);
            }
            store_columns<GATHER>(p, t.store_bytes, v, turn, slot, mine - q * 32, live,
                                  n0 + quarter * 32, lane);
          }
        }
      } else {
        // the other CTAs have read this one's last part
        ok = tc_wait_warp<true>(part_empty, (nt & 1) ^ 1, abort_flag, p.err, kErrTcJoin);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < Sh::kWarpCols / 2; ++i) {
          float* to = part + (cols0 + 2 * i) * kPartPitch + quarter * 32 + lane;
          to[0] = __uint_as_float((uint32_t)acc[i]);
          to[kPartPitch] = __uint_as_float((uint32_t)(acc[i] >> 32));
        }
        __syncwarp();
        if (lane < csize) tc::mbar_arrive_cluster(tc::map_rank(part_full, lane));
        ok = tc_wait_warp<true>(part_full, nt & 1, abort_flag, p.err, kErrTcJoin);
        if (!ok) break;
        // each CTA sums its share of the tile, four weights to a thread, the
        // parts in rank order
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
    const uint32_t bar0 = tc::map_rank(full0, CG == 2 ? 0 : rank);
    RingPos at;
    uint32_t armed = 0;        // stages given to TMA, all but the last NS done
    bool ok = true;
    if (p.stall_test && blockIdx.x == 0)
      ok = tc_wait_warp<false>(tc::smem_addr(&bb->never), 0, abort_flag, p.err, kErrTcEmpty);
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      int boxes = 0;           // of slots' rows, per CTA
#pragma unroll
      for (int h = 0; h < Sh::kHalves; ++h)
        boxes += (half_slots<Sh>(w, h) / CG + kF8Box - 1) / kF8Box;
      const uint32_t bytes = CG * (Sh::kABytes + (GATHER ? 0 : boxes * kF8Box * kTcRowBytes));
      const int n0 = w.wt * kTileWeights + w_rank * kTcWeights;
      for (int c = c0; c < c1; ++c, at.next(NS), ++armed) {
        const uint32_t s = at.stage;
        ok = tc_wait_warp<kPair>(empty0 + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        if (tc::elect_one()) {
          if (w_rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, bytes);
          tc::load_3d<CG>(base + s * Sh::kStageBytes, &map_w, c * kTcRowBytes, n0, w.e,
                          bar0 + 8 * s);
        }
        __syncwarp();
      }
    }
    // After an abort: the stages in flight land before the CTA leaves.
    if (*abort_flag && w_rank == 0) {
      for (uint32_t k = armed > NS ? armed - NS : 0; k < armed; ++k) {
        const uint64_t begin = globaltimer_ns();
        while (!tc::mbar_wait_some<true>(full0 + 8 * (k % NS), (k / NS) & 1, kTcSleepNs) &&
               globaltimer_ns() - begin < kWaitLimitNs) {}
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------- matrix instructions
    if (w_rank == 0) {
      RingPos at;
      uint32_t nb[2] = {0, 0};             // blocks of each half so far
      bool ok = true;
      const uint64_t desc0 = tc::operand_desc(base);
      for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
        const Tile w = find_tile(g, p.E, tile, wts, BN);
        uint32_t idesc[2] = {0u, 0u};
#pragma unroll
        for (int h = 0; h < Sh::kHalves; ++h)
          if (half_slots<Sh>(w, h) > 0)
            idesc[h] = tc::idesc_e4m3(kTileWeights, half_slots<Sh>(w, h));
        for (int c = 0; ok && c < nc; ++c, at.next(NS)) {
          const uint32_t s = at.stage;
          ok = tc_wait_warp<kPair>(full0 + 8 * s, at.phase, abort_flag, p.err, kErrTcFull);
          if (!ok) break;
          const uint64_t da = desc0 + (s * Sh::kStageBytes >> 4);
#pragma unroll
          for (int h = 0; h < Sh::kHalves; ++h) {
            if (idesc[h] == 0u) continue;
            const uint32_t b = nb[h] & 1;
            ok = ok && tc_wait_warp<kPair>(aempty0 + (b * 2 + h) * 8, ((nb[h] >> 1) & 1) ^ 1,
                                           abort_flag, p.err, kErrTcTile);
            if (!ok) break;
            tc::fence_after();
            const uint64_t db =
                da + ((Sh::kABytes + h * (Sh::kHalf / CG) * kTcRowBytes) >> 4);
            const uint32_t d = tmem + b * BN + h * Sh::kHalf;
            if (tc::elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc::mma_fp8<CG>(d, da + 2 * k, db + 2 * k, idesc[h], k > 0 ? 1u : 0u);
              tc::commit<CG>(afull0 + (b * 2 + h) * 8);
            }
            ++nb[h];
          }
          if (!ok) break;
          if (tc::elect_one()) tc::commit<CG>(empty0 + 8 * s);
        }
      }
    }
    __syncwarp();
  } else if (warp == 11 || warp == 12) {
    // -------------------------------------------------------------- scales
    // Lane l has the slots l, l + 32, ... of its warp's part of the columns;
    // sa * sb, the block's slots one after the other.
    const int first = (warp - 11) * (BN / kF8ScaleWarps);
    float* to0 = reinterpret_cast<float*>(smem + t.scales_at) + first;
    uint32_t ng = 0;
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      const float* row[Sh::kLaneSlots];
#pragma unroll
      for (int i = 0; i < Sh::kLaneSlots; ++i) {
        const int s = first + i * 32 + lane;
        row[i] = nullptr;
        if (s < w.n) {
          int64_t r = (int64_t)w.slot0 + s;
          if constexpr (GATHER) r = p.rows[r];
          if (r >= 0 && r < p.n_a) row[i] = t.a_scale + r * t.HB;
        }
      }
      const int64_t wb = (int64_t)w.wt * CG + w_rank;
      const float* sb = wb < t.NB ? t.b_scale + ((int64_t)w.e * t.NB + wb) * t.HB : nullptr;
      for (int c = c0; c < c1; c += kF8ScaleBlocks, ++ng) {
        const int have = min(kF8ScaleBlocks, c1 - c);
        float v[Sh::kLaneSlots][kF8ScaleBlocks], vb[kF8ScaleBlocks];
#pragma unroll
        for (int j = 0; j < kF8ScaleBlocks; ++j) vb[j] = sb && j < have ? __ldg(sb + c + j) : 0.0f;
#pragma unroll
        for (int i = 0; i < Sh::kLaneSlots; ++i) {
          if (t.scale_vec && row[i] && have == kF8ScaleBlocks && (c & 3) == 0) {
            const float4 u = __ldg(reinterpret_cast<const float4*>(row[i] + c));
            v[i][0] = u.x; v[i][1] = u.y; v[i][2] = u.z; v[i][3] = u.w;
          } else {
#pragma unroll
            for (int j = 0; j < kF8ScaleBlocks; ++j)
              v[i][j] = row[i] && j < have ? __ldg(row[i] + c + j) : 0.0f;
          }
        }
        const uint32_t slot = ng % kF8ScaleSlots;
        ok = tc_wait_warp<false>(sempty0 + 8 * slot, (ng / kF8ScaleSlots & 1) ^ 1, abort_flag,
                                 p.err, kErrTcEmpty);
        if (!ok) break;
        float* to = to0 + slot * (Sh::kScaleSlot / 4) + lane;
#pragma unroll
        for (int i = 0; i < Sh::kLaneSlots; ++i)
#pragma unroll
          for (int j = 0; j < kF8ScaleBlocks; ++j) to[j * BN + i * 32] = v[i][j] * vb[j];
        __syncwarp();
        if (lane == 0) mbar_arrive(sfull0 + 8 * slot);
      }
    }
  } else if (!GATHER && warp == 10) {
    // --------------------------------------------------- slots' producer
    const uint32_t bar0 = tc::map_rank(full0, CG == 2 ? 0 : rank);
    RingPos at;
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      for (int c = c0; c < c1; ++c, at.next(NS)) {
        const uint32_t s = at.stage;
        ok = tc_wait_warp<kPair>(empty0 + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        const uint32_t b = base + s * Sh::kStageBytes + Sh::kABytes;
        if (tc::elect_one()) {
#pragma unroll
          for (int h = 0; h < Sh::kHalves; ++h) {
            const int rows = half_slots<Sh>(w, h) / CG;
            const int first = w.slot0 + h * Sh::kHalf + w_rank * rows;
#pragma unroll
            for (int i = 0; i < Sh::kHalf / CG / kF8Box; ++i)
              if (i * kF8Box < rows)
                tc::load_2d<CG>(b + (h * (Sh::kHalf / CG) + i * kF8Box) * kTcRowBytes, &map_x,
                                c * kTcRowBytes, first + i * kF8Box, bar0 + 8 * s);
          }
        }
        __syncwarp();
      }
    }
  } else if (GATHER && (warp == 10 || warp >= 13)) {
    // -------------------------------------------------------- gathered rows
    // A warp takes every fourth stage.  Eight lanes copy a row's 128 bytes, in
    // the swizzled layout that TMA would write: 16-byte column j of row r at
    // j ^ (r & 7).  Lane l knows the rows l, l + 32, ...
    constexpr int kHeld = Sh::kRows / 32, kPer = Sh::kHalf / CG / 32;    // per half
    const int mine = warp == 10 ? 0 : warp - 12, col = lane & 7, sub = lane >> 3;
    const char* x = static_cast<const char*>(p.a) + col * 16;
    const uint64_t pitch = (uint64_t)p.H;
    RingPos at;
    at.skip(mine, NS);
    int ahead = mine;
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      int32_t held[kHeld];                   // negative: zeros
      int rows[Sh::kHalves];
#pragma unroll
      for (int h = 0; h < Sh::kHalves; ++h) rows[h] = half_slots<Sh>(w, h) / CG;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int h = i / kPer, in = (i % kPer) * 32 + lane;
        const int s = h * Sh::kHalf + w_rank * rows[h] + in;
        held[i] = -1;
        if (in < rows[h] && s < w.n) held[i] = p.rows[(int64_t)w.slot0 + s];
        if (held[i] >= p.n_a) held[i] = -1;
      }
      int c = c0 + ahead;
      for (; c < c1; c += kF8Gather, at.skip(kF8Gather, NS)) {
        const uint32_t s = at.stage;
        ok = tc_wait_warp<kPair>(empty0 + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        const uint32_t b = base + s * Sh::kStageBytes + Sh::kABytes + sub * kTcRowBytes;
        const bool in_row = (int64_t)c * kTcRowBytes + col * 16 < p.H;
        const char* from = x + (int64_t)c * kTcRowBytes;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {       // rows i * 32 + j * 4 + sub
            if ((i % kPer) * 32 + j * 4 >= rows[i / kPer]) break;
            const int32_t row = __shfl_sync(0xFFFFFFFFu, held[i], j * 4 + sub);
            const bool have = in_row && row >= 0;
            tc::copy16(b + (i * 32 + j * 4) * kTcRowBytes + ((col ^ ((j * 4 + sub) & 7)) << 4),
                       have ? from + (uint32_t)row * pitch : p.a, have ? 16u : 0u);
          }
        cp_async_commit();
        cp_async_wait<0>();
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_first<CG>(full0 + 8 * s);
      }
      ahead = c - c1;
    }
  }

  // As in farn_product_tc_kernel: after an abort the tensor cores may still be
  // at work on what they were given.
  __syncthreads();
  if (*abort_flag && warp == 9 && w_rank == 0) {
    const uint32_t never = tc::smem_addr(&bb->never);
    if (tc::elect_one()) tc::commit<CG>(never);
    __syncwarp();
    const uint64_t begin = globaltimer_ns();
    while (!tc::mbar_wait_some<true>(never, 0, kTcSleepNs) &&
           globaltimer_ns() - begin < kWaitLimitNs) {}
  }
  tc::fence_before();
  if (csize > 1) tc::cluster_sync(); else __syncthreads();
  tc::fence_after();
  if (warp == 9) tc::tmem_free<CG>(tmem, Sh::kCols);
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
          vb = e4m3_to_f32(static_cast<const uint8_t*>(p.b)[((int64_t)w.e * p.N + n0 + r) * p.H + h]);
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

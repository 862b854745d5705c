// The products on the tensor cores.
//
// The weights are the matrix instruction's M side (128 rows per CTA) and the
// slots its N side, so that a tile's slots can be any multiple of 16 up to
// BN: a group's ragged end costs what it has, and a decoding batch of a few
// rows still streams full tiles of weights.  The accumulator is transposed
// on the way out.
//
// A CTA has a producer warp (TMA), a warp that issues the matrix
// instructions, four epilogue warps, and for NVFP4 four warps that bring the
// block scales into the layout the tensor cores read, or for a gathering call
// four warps that copy the slots' rows (cp.async: a TMA gather of four rows of
// 128 bytes took 95 cycles, 3 times the matrix instructions' time).  The ring of stages runs on across
// tiles, and two accumulators let the epilogue of one tile overlap the
// products of the next.
//
//   CG = 2  pairs of CTAs share a tile of 256 weights, each holding half of
//           the slots' rows: long calls, bound by the tensor cores
//   CG = 1  one CTA per tile of 128 weights; `ks` CTAs of a cluster may split
//           the row and join their accumulators, in rank order, through
//           distributed shared memory: short calls, bound by reading weights
//
// Every wait is bounded (see wait_phase); a CTA that gives up sets its bit in
// the status word, waits for its own copies and leaves.
#pragma once

#include <cuda.h>

#include "farn_product.cuh"
#include "farn_tcgen05.cuh"

namespace farn {

constexpr int kTcMaxStages = 12;
constexpr int kTcRowBytes = 128;       // bytes of a row per stage: one swizzle span
constexpr int kTcWeights = 128;        // weights per CTA and tile
constexpr int kTcWarpsBf16 = 6;
// Further warps for block scales, or for gathered rows.  Each takes every
// kAux-th stage.  They may not be more than the ring has stages: a warp that
// waits for a stage has to be within one round of the ring, or the parity of
// the phase it waits for says nothing.
constexpr int kTcAuxFp4 = 4;
constexpr int kTcAuxGather = 6;
constexpr int kTcWarpsMost = kTcWarpsBf16 + kTcAuxGather;
constexpr int kErrTcFull = 16;         // status bits: matrix warp waiting for operands,
constexpr int kErrTcEmpty = 32;        // producers waiting for a free stage,
constexpr int kErrTcTile = 64;         // epilogue or matrix warp waiting for a tile,
constexpr int kErrTcJoin = 128;        // epilogue waiting for the other parts of the row

struct TcParams {
  ProductParams p;
  int stages;
  int ks;            // CTAs of a cluster that split the row (CG = 1)
  int pair_stores;   // N even and out 4-byte aligned
  int tma_scales;    // NVFP4: rows of scales that TMA can read, else
  int scale_step;    // bytes per load of scales that alignment allows
  uint32_t groups_at;  // shared-memory offsets
  uint32_t part_at;    // fp32 [BN][kPartPitch], for ks > 1
};

struct TcBarriers {
  uint64_t full[kTcMaxStages];
  uint64_t raw[kTcMaxStages];      // block scales as they lie in memory
  uint64_t empty[kTcMaxStages];
  uint64_t tile_full[2];
  uint64_t tile_empty[2];
  uint64_t part_full;
  uint64_t part_empty;
  uint64_t never;          // nothing arrives on it (stall_test)
  uint32_t tmem;
  int abort_flag;
};

constexpr int kPartPitch = kTcWeights + 4;

template <bool FP4, int CG, int BN, bool GATHER>
struct TcShape {
  static constexpr int kAux = FP4 ? kTcAuxFp4 : GATHER ? kTcAuxGather : 0;
  static constexpr int kWarps = kTcWarpsBf16 + kAux;
  static constexpr int kRows = BN / CG;                      // slots per CTA
  static constexpr int kBox = kRows % 32 == 0 ? 32 : 16;     // rows of a TMA box
  static constexpr int kABytes = kTcWeights * kTcRowBytes;
  static constexpr int kBBytes = kRows * kTcRowBytes;
  static constexpr int kSlotBlocks = (BN + 127) / 128;       // blocks of 128 slots' scales
  static constexpr int kScaleBytes = FP4 ? 2048 * (1 + kSlotBlocks) : 0;
  static constexpr int kStageBytes = kABytes + kBBytes + kScaleBytes;
  static constexpr int kScaleCols = FP4 ? 16 * (1 + kSlotBlocks) : 0;
  static constexpr int kColsUsed = 2 * BN + kScaleCols;
  static constexpr int kCols = kColsUsed <= 32 ? 32 : kColsUsed <= 64 ? 64
                               : kColsUsed <= 128 ? 128 : kColsUsed <= 256 ? 256 : 512;
  static constexpr int kChunk = FP4 ? 256 : 64;              // elements of a row per stage
  static constexpr int kStep = 16 * CG;                      // granularity of a tile's slots
  static_assert(kColsUsed <= 512 && kBBytes % 1024 == 0 && kScaleBytes % 1024 == 0, "");
};

// Bounded phase wait.  JOIN: what other CTAs of the cluster wrote before they
// arrived is read afterwards.
constexpr uint32_t kTcSleepNs = 1000000;

template <bool JOIN = false>
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                        int* err, int code) {
  if (tc::mbar_wait_some<JOIN>(bar, parity, kTcSleepNs)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (tc::mbar_wait_some<JOIN>(bar, parity, kTcSleepNs)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      atomicOr(err, code);
      return false;
    }
  }
}

// A place in the ring of stages.
struct RingPos {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++stage == stages) { stage = 0; phase ^= 1; }
  }
  // `by` stages on
  __device__ __forceinline__ void skip(uint32_t by, uint32_t stages) {
    for (stage += by; stage >= stages; stage -= stages) phase ^= 1;
  }
};

// The same by a whole warp, whose lanes go on or give up together.
template <bool JOIN = false>
__device__ __forceinline__ bool tc_wait_warp(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag, int* err, int code) {
  return __all_sync(0xFFFFFFFFu, tc_wait<JOIN>(bar, parity, abort_flag, err, code));
}

// 16 scale bytes of a row from `at`, of which `left` belong to the row; the
// rest are 0.
__device__ __forceinline__ uint4 load_scales16(const uint8_t* at, int64_t left, int step) {
  if (step == 16 && left >= 16) return __ldg(reinterpret_cast<const uint4*>(at));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (step >= 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * i < left) w[i] = __ldg(reinterpret_cast<const uint32_t*>(at) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) w[i >> 2] |= (uint32_t)__ldg(at + i) << (8 * (i & 3));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool FP4, int CG, int BN, bool GATHER>
__global__ void __launch_bounds__(TcShape<FP4, CG, BN, GATHER>::kWarps * 32, 1)
farn_product_tc_kernel(const __grid_constant__ TcParams t,
                       const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ CUtensorMap map_x,
                       const __grid_constant__ CUtensorMap map_part,
                       const __grid_constant__ CUtensorMap map_ws,
                       const __grid_constant__ CUtensorMap map_xs) {
  using Sh = TcShape<FP4, CG, BN, GATHER>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const ProductParams& p = t.p;
  const uint32_t base = (tc::smem_addr(smem_raw) + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - tc::smem_addr(smem_raw));
  const uint32_t NS = t.stages;
  TcBarriers* bb = reinterpret_cast<TcBarriers*>(smem + (size_t)NS * Sh::kStageBytes);
  const Groups g = groups_at(smem + t.groups_at, p.E);
  const uint32_t full0 = tc::smem_addr(&bb->full[0]);
  const uint32_t empty0 = tc::smem_addr(&bb->empty[0]);
  const uint32_t raw0 = tc::smem_addr(&bb->raw[0]);
  const uint32_t tfull0 = tc::smem_addr(&bb->tile_full[0]);
  const uint32_t tempty0 = tc::smem_addr(&bb->tile_empty[0]);
  volatile int* abort_flag = &bb->abort_flag;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // uniform
  const uint32_t rank = cluster_ctarank();
  const int csize = CG == 2 ? 2 : t.ks;

  if (tid == 0) {
    for (uint32_t s = 0; s < NS; ++s) {
      mbar_init(full0 + 8 * s, Sh::kAux ? 1 + CG : 1);   // TMA; scales or gathered rows
      mbar_init(empty0 + 8 * s, 1);
      mbar_init(raw0 + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull0 + 8 * i, 1);
      mbar_init(tempty0 + 8 * i, 4 * CG);
    }
    mbar_init(tc::smem_addr(&bb->part_full), 4 * csize);
    mbar_init(tc::smem_addr(&bb->part_empty), 4 * csize);
    mbar_init(tc::smem_addr(&bb->never), 1);
    bb->abort_flag = 0;
    tc::mbar_init_fence();
  }
  if (warp == 5) tc::tmem_alloc<CG>(tc::smem_addr(&bb->tmem), Sh::kCols);
  if (tid == 4 * 32) {
    tc::prefetch_map(&map_w);
    if constexpr (!GATHER) {
      tc::prefetch_map(&map_x);
      tc::prefetch_map(&map_part);
    }
    if (FP4 && t.tma_scales) {
      tc::prefetch_map(&map_ws);
      tc::prefetch_map(&map_xs);
    }
  }
  pdl_wait();
  pdl_trigger();
  load_groups(g, p, BN);            // ends with a block barrier
  tc::fence_before();
  if (csize > 1) tc::cluster_sync(); else __syncthreads();
  tc::fence_after();
  const uint32_t tmem = bb->tmem;

  constexpr int kTileWeights = kTcWeights * CG;
  const int wts = (int)((p.N + kTileWeights - 1) / kTileWeights);
  const int64_t tiles = (int64_t)g.tile[p.E] * wts;
  const int64_t t0 = blockIdx.x / csize, tstep = gridDim.x / csize;
  const int chunks = (int)((p.H + Sh::kChunk - 1) / Sh::kChunk);
  const int c0 = CG == 2 ? 0 : (int)((int64_t)chunks * rank / csize);
  const int c1 = CG == 2 ? chunks : (int)((int64_t)chunks * (rank + 1) / csize);
  const int nc = c1 - c0;
  const int w_rank = CG == 2 ? (int)rank : 0;      // this CTA's part of a tile's weights

  if (warp == 4) {
    // ---------------------------------------------------------- producer
    const uint32_t bar_rank = CG == 2 ? 0 : rank;
    RingPos at;
    uint32_t armed = 0;        // stages given to TMA, all but the last NS done
    bool ok = true;
    if (t.p.stall_test && blockIdx.x == 0)
      ok = tc_wait_warp(tc::smem_addr(&bb->never), 0, abort_flag, p.err, kErrTcEmpty);
    for (int64_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      const int n_eff = (w.n + Sh::kStep - 1) / Sh::kStep * Sh::kStep;
      const int rows = n_eff / CG;                       // of this CTA, a multiple of 16
      const int first = w.slot0 + w_rank * rows;
      // whole tiles with one box, others with boxes of a few rows
      const bool whole = rows > Sh::kRows - Sh::kBox;
      const int loads = GATHER ? 0 : whole ? 1 : (rows + Sh::kBox - 1) / Sh::kBox;
      const uint32_t bytes = (uint32_t)loads * (whole ? Sh::kRows : Sh::kBox) * kTcRowBytes;
      const int n0 = w.wt * kTileWeights + w_rank * kTcWeights;
      for (int c = c0; c < c1; ++c, at.next(NS), ++armed) {
        const uint32_t s = at.stage;
        ok = tc_wait_warp(empty0 + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        const uint32_t a = base + s * Sh::kStageBytes, b = a + Sh::kABytes;
        const uint32_t bar = tc::map_rank(full0 + 8 * s, bar_rank);
        const int x = c * (FP4 ? kTcRowBytes : Sh::kChunk);
        if (tc::elect_one()) {
          if (w_rank == 0)
            mbar_arrive_expect_tx(full0 + 8 * s, CG * (Sh::kABytes + bytes));
          tc::load_3d<CG>(a, &map_w, x, n0, w.e, bar);
          if (!GATHER && whole) {
            tc::load_2d<CG>(b, &map_x, x, first, bar);
          } else if constexpr (!GATHER) {
            for (int i = 0; i < loads; ++i)
              tc::load_2d<CG>(b + i * Sh::kBox * kTcRowBytes, &map_part, x, first + i * Sh::kBox,
                              bar);
          }
          if (FP4 && t.tma_scales) {
            const int blocks = w.n > 128 ? 2 : 1;
            const uint32_t sc = b + Sh::kBBytes, rbar = raw0 + 8 * s;
            mbar_arrive_expect_tx(rbar, 2048 * (1 + blocks));
            tc::load_2d<1>(sc, &map_ws, c * 16, n0, rbar);
            tc::load_2d<1>(sc + 2048, &map_xs, c * 16, w.slot0, rbar);
            if (blocks > 1) tc::load_2d<1>(sc + 4096, &map_xs, c * 16, w.slot0 + 128, rbar);
          }
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
  } else if (warp == 5) {
    // ------------------------------------------------- matrix instructions
    if (w_rank == 0) {
      RingPos at;
      uint32_t nt = 0;
      bool ok = true;
      const uint64_t desc0 = tc::operand_desc(base);
      const uint64_t scale0 = tc::scale_desc(base + Sh::kABytes + Sh::kBBytes);
      const uint32_t sf_a = tmem + 2 * BN, sf_b = sf_a + 16;
      for (int64_t tile = t0; ok && tile < tiles; tile += tstep, ++nt) {
        const Tile w = find_tile(g, p.E, tile, wts, BN);
        const int n_eff = (w.n + Sh::kStep - 1) / Sh::kStep * Sh::kStep;
        const uint32_t idesc = FP4 ? tc::idesc_nvfp4(kTileWeights, n_eff)
                                   : tc::idesc_bf16(kTileWeights, n_eff);
        const uint32_t acc = nt & 1, d = tmem + acc * BN;
        ok = tc_wait_warp(tempty0 + 8 * acc, ((nt >> 1) & 1) ^ 1, abort_flag, p.err, kErrTcTile);
        if (!ok) break;
        tc::fence_after();
        for (int c = 0; c < nc; ++c, at.next(NS)) {
          const uint32_t s = at.stage, ph = at.phase;
          ok = tc_wait_warp(full0 + 8 * s, ph, abort_flag, p.err, kErrTcFull);
          if (!ok) break;
          tc::fence_after();
          const uint64_t da = desc0 + (s * Sh::kStageBytes >> 4), db = da + (Sh::kABytes >> 4);
          if (tc::elect_one()) {
          if constexpr (FP4) {
            const uint64_t sc = scale0 + (s * Sh::kStageBytes >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              tc::copy_scales<CG>(sf_a + 4 * k, sc + (512 >> 4) * k);
#pragma unroll
              for (int j = 0; j < Sh::kSlotBlocks; ++j)
                if (j == 0 || n_eff > 128)
                  tc::copy_scales<CG>(sf_b + (k * Sh::kSlotBlocks + j) * 4,
                                      sc + (2048 >> 4) * (1 + j) + (512 >> 4) * k);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_nvfp4<CG>(d, da + 2 * k, db + 2 * k, idesc, sf_a + 4 * k,
                                sf_b + 4 * k * Sh::kSlotBlocks, c > 0 || k > 0);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_bf16<CG>(d, da + 2 * k, db + 2 * k, idesc, c > 0 || k > 0);
          }
          tc::commit<CG>(empty0 + 8 * s);
          if (c == nc - 1) tc::commit<CG>(tfull0 + 8 * acc);
          }
          __syncwarp();
        }
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------- epilogue
    uint32_t nt = 0;
    bool ok = true;
    uint16_t* out = static_cast<uint16_t*>(p.out);
    const uint32_t part_full = tc::smem_addr(&bb->part_full);
    const uint32_t part_empty = tc::smem_addr(&bb->part_empty);
    float* part = reinterpret_cast<float*>(smem + t.part_at);
    for (int64_t tile = t0; ok && tile < tiles; tile += tstep, ++nt) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      const uint32_t acc = nt & 1, d = tmem + acc * BN + ((uint32_t)warp << 21);
      const int64_t n0 = (int64_t)w.wt * kTileWeights + w_rank * kTcWeights;
      ok = tc_wait_warp(tfull0 + 8 * acc, (nt >> 1) & 1, abort_flag, p.err, kErrTcTile);
      if (!ok) break;
      tc::fence_after();
      const bool split = CG == 1 && csize > 1;
      if (split) {
        // the other CTAs have read this one's last part
        ok = tc_wait_warp<true>(part_empty, (nt & 1) ^ 1, abort_flag, p.err, kErrTcJoin);
        if (!ok) break;
        for (int c = 0; c < w.n; c += 16) {
          uint32_t v[16];
          tc::tmem_ld16(d + c, v);
          tc::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            part[(c + j) * kPartPitch + warp * 32 + lane] = __uint_as_float(v[j]);
        }
      } else {
        const int64_t n = n0 + warp * 32 + lane;
        for (int c = 0; c < w.n; c += 16) {
          uint32_t v[16];
          tc::tmem_ld16(d + c, v);
          uint32_t live = 0xFFFFu;
          if constexpr (GATHER) {
            const int64_t s = (int64_t)w.slot0 + c + lane;
            const int r = lane < 16 && c + lane < w.n ? p.rows[s] : -1;
            live = __ballot_sync(0xFFFFFFFFu, r >= 0 && r < p.n_a);
          }
          tc::tmem_ld_wait();
          if (t.pair_stores) {
            // lanes 2i and 2i + 1 exchange halves: the even one stores slots
            // 0..7 of both weights, the odd one slots 8..15
            const bool odd = lane & 1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float keep = __uint_as_float(odd ? v[j + 8] : v[j]);
              const float send = __uint_as_float(odd ? v[j] : v[j + 8]);
              const float got = __shfl_xor_sync(0xFFFFFFFFu, send, 1);
              const int jj = j + (odd ? 8 : 0);
              uint32_t word = pack_bf16x2((odd ? got : keep) * p.alpha,
                                          (odd ? keep : got) * p.alpha);
              if (!((live >> jj) & 1u)) word = 0u;
              if (c + jj < w.n && n < p.N)
                *reinterpret_cast<uint32_t*>(
                    out + ((int64_t)w.slot0 + c + jj) * p.N + (n & ~(int64_t)1)) = word;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < w.n && n < p.N)
                out[((int64_t)w.slot0 + c + j) * p.N + n] =
                    (live >> j) & 1u ? to_bf16(__uint_as_float(v[j]) * p.alpha) : (uint16_t)0;
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(tc::map_rank(tempty0 + 8 * acc, CG == 2 ? 0 : rank));
      if (split) {
        if (lane < csize) tc::mbar_arrive_cluster(tc::map_rank(part_full, lane));
        ok = tc_wait_warp<true>(part_full, nt & 1, abort_flag, p.err, kErrTcJoin);
        if (!ok) break;
        const uint32_t mine = tc::smem_addr(part);
        for (int i = (int)rank * 128 + tid; i < w.n * 128; i += csize * 128) {
          const int j = i >> 7, k = i & 127;
          float sum = 0.0f;
          for (int q = 0; q < csize; ++q)
            sum += tc::ld_cluster_f32(tc::map_rank(mine, q) + (j * kPartPitch + k) * 4);
          const int64_t s = (int64_t)w.slot0 + j;
          bool live = true;
          if constexpr (GATHER) live = p.rows[s] >= 0 && p.rows[s] < p.n_a;
          if (n0 + k < p.N) out[s * p.N + n0 + k] = live ? to_bf16(sum * p.alpha) : (uint16_t)0;
        }
        __syncwarp();
        if (lane < csize) tc::mbar_arrive_cluster(tc::map_rank(part_empty, lane));
      }
    }
  } else if constexpr (FP4) {
    // ------------------------------------------------------- block scales
    // Warp i takes every fourth stage.  A lane reads 16 bytes (256 elements)
    // of rows lane, +32, +64 and +96 of a block of 128 and writes them
    // transposed: word r of the lane's 16 bytes of atom k is row lane + 32 r's
    // four scales of the k-th 64 elements.
    const int mine = warp - 6;
    const int64_t pitch = p.H / 16;
    RingPos at;
    at.skip(mine, NS);
    int ahead = mine;          // stages until this warp's next
    bool ok = true;
    for (int64_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      const int64_t n0 = (int64_t)w.wt * kTileWeights + w_rank * kTcWeights;
      const int blocks = (w.n + 127) / 128;
      int c = c0 + ahead;
      for (; c < c1; c += Sh::kAux, at.skip(Sh::kAux, NS)) {
        const uint32_t s = at.stage;
        const int64_t left = pitch - (int64_t)c * 16;
        uint4 v[1 + Sh::kSlotBlocks][4];
        unsigned char* dst = smem + s * Sh::kStageBytes + Sh::kABytes + Sh::kBBytes;
        if (t.tma_scales) {
          ok = tc_wait_warp(raw0 + 8 * s, at.phase, abort_flag, p.err, kErrTcFull);
          if (!ok) break;
#pragma unroll
          for (int u = 0; u <= Sh::kSlotBlocks; ++u) {
            if (u > blocks) break;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              v[u][r] = reinterpret_cast<const uint4*>(dst + u * 2048)[r * 32 + lane];
          }
          __syncwarp();       // in place: all of it is read before any is written
        } else {
#pragma unroll
        for (int u = 0; u <= Sh::kSlotBlocks; ++u) {
          if (u > blocks) break;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int in = (u ? (u - 1) * 128 : 0) + r * 32 + lane;
            const bool have = u ? in < w.n : n0 + in < p.N;
            const int64_t row = u ? (int64_t)w.slot0 + in : (int64_t)w.e * p.N + n0 + in;
            v[u][r] = have ? load_scales16((u ? p.a_scale : p.b_scale) + row * pitch + c * 16,
                                           left, t.scale_step)
                           : make_uint4(0u, 0u, 0u, 0u);
          }
        }
        ok = tc_wait_warp(empty0 + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        }
#pragma unroll
        for (int u = 0; u <= Sh::kSlotBlocks; ++u) {
          if (u > blocks) break;
          uint4* at = reinterpret_cast<uint4*>(dst + u * 2048) + lane;
          at[0] = make_uint4(v[u][0].x, v[u][1].x, v[u][2].x, v[u][3].x);
          at[32] = make_uint4(v[u][0].y, v[u][1].y, v[u][2].y, v[u][3].y);
          at[64] = make_uint4(v[u][0].z, v[u][1].z, v[u][2].z, v[u][3].z);
          at[96] = make_uint4(v[u][0].w, v[u][1].w, v[u][2].w, v[u][3].w);
        }
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(tc::map_rank(full0 + 8 * s, CG == 2 ? 0 : rank));
      }
      ahead = c - c1;
    }
  }

  if constexpr (GATHER) {
    if (warp >= 6) {
      // ------------------------------------------------------ gathered rows
      // Warp i takes every sixth stage, so that a stage's copies have the whole
      // ring's time to land.  Eight lanes copy a row's 128 bytes, in the
      // swizzled layout that TMA would write: 16-byte column j of row r at
      // j ^ (r & 7).  Lane l knows the rows l, l + 32, l + 64 and l + 96.
      constexpr int kHeld = (Sh::kRows + 31) / 32;
      const int mine = warp - 6, col = lane & 7, sub = lane >> 3;
      const char* x = static_cast<const char*>(p.a) + col * 16;
      const uint64_t pitch = (uint64_t)p.H * 2;
      RingPos at;
      at.skip(mine, NS);
      int ahead = mine;
      bool ok = true;
      for (int64_t tile = t0; ok && tile < tiles; tile += tstep) {
        const Tile w = find_tile(g, p.E, tile, wts, BN);
        const int n_eff = (w.n + Sh::kStep - 1) / Sh::kStep * Sh::kStep;
        const int rows = n_eff / CG;           // a multiple of 16
        int32_t held[kHeld];                   // negative: zeros
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          const int r = w_rank * rows + i * 32 + lane;
          held[i] = -1;
          if (i * 32 + lane < rows && r < w.n) held[i] = p.rows[(int64_t)w.slot0 + r];
          if (held[i] >= p.n_a) held[i] = -1;
        }
        int c = c0 + ahead;
        for (; c < c1; c += Sh::kAux, at.skip(Sh::kAux, NS)) {
          const uint32_t s = at.stage;
          ok = tc_wait_warp(empty0 + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
          if (!ok) break;
          const uint32_t b = base + s * Sh::kStageBytes + Sh::kABytes + sub * kTcRowBytes;
          const bool in_row = (int64_t)c * Sh::kChunk + col * 8 < p.H;
          const char* from = x + (int64_t)c * kTcRowBytes;
#pragma unroll
          for (int i = 0; i < kHeld; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {       // rows i * 32 + j * 4 + sub
              if (i * 32 + j * 4 >= rows) break;
              const int32_t row = __shfl_sync(0xFFFFFFFFu, held[i], j * 4 + sub);
              const bool have = in_row && row >= 0;
              tc::copy16(b + (i * 32 + j * 4) * kTcRowBytes + ((col ^ ((j * 4 + sub) & 7)) << 4),
                         have ? from + (uint32_t)row * pitch : p.a, have ? 16u : 0u);
            }
          cp_async_commit();
          cp_async_wait<0>();
          tc::fence_async_shared();
          __syncwarp();
          if (lane == 0)
            tc::mbar_arrive_cluster(tc::map_rank(full0 + 8 * s, CG == 2 ? 0 : rank));
        }
        ahead = c - c1;
      }
    }
  }

  // The matrix warp's last commits have arrived when the epilogue is done
  // with the last tile; after an abort the tensor cores may still be at work
  // on what they were given, so the warp waits for that here.
  __syncthreads();
  if (*abort_flag && warp == 5 && w_rank == 0) {
    const uint32_t never = tc::smem_addr(&bb->never);
    if (tc::elect_one()) tc::commit<CG>(never);
    __syncwarp();
    const uint64_t begin = globaltimer_ns();
    while (!tc::mbar_wait_some<true>(never, 0, kTcSleepNs) && globaltimer_ns() - begin < kWaitLimitNs) {}
  }
  tc::fence_before();
  if (csize > 1) tc::cluster_sync(); else __syncthreads();
  tc::fence_after();
  if (warp == 5) tc::tmem_free<CG>(tmem, Sh::kCols);
}

}  // namespace farn

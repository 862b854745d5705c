// The products on the tensor cores.
//
// The weights are the matrix instruction's M side (128 rows per CTA) and the
// slots its N side, so that a tile's slots can be any multiple of 16 (32) up
// to BN: a group's ragged end costs what it has, and a decoding batch of a few
// rows still streams full tiles of weights.  The accumulator is turned over on
// the way out.
//
//   CG = 2  pairs of CTAs share a tile of 256 weights by 256 slots (NVFP4:
//           224, so that two accumulators and the scales fit the tensor
//           memory), each holding half of the slots' rows: long calls
//   CG = 1  one CTA per tile of 128 weights by 64 slots; up to four CTAs of a
//           cluster split the row and join their accumulators, in rank order,
//           through distributed shared memory: short calls
//
// Warps of a CTA: four for the epilogue, one that has TMA fetch the weights,
// one that issues the matrix instructions, one that has TMA fetch the slots'
// rows; or, for a gathering call, six that copy the rows themselves (a TMA
// gather of four rows of 128 bytes took 95 cycles, three times the matrix
// instructions' time); for NVFP4 also those that bring the block scales into
// the layout the tensor cores read.  The ring of stages (128 bytes of every
// row) runs on across tiles, and two accumulators let the epilogue of one tile
// overlap the products of the next.
//
// What bounds it (GB300, us and rates of the kernel alone): bf16 8192^3 takes
// 564 us (1.95 PFLOP/s, 101 % of the measured library rate) with the tensor
// pipe 92 % busy, under the power limit; NVFP4 8192^3 173 us (6.35 PFLOP/s; 195
// to 200 us in a row of calls, where the power limit lowers the clock), 69 %
// busy: a stage's synchronisation takes about 600 cycles, its products 450.
// 64 experts of 64 tokens, 2048 -> 7168: 280 us, the weights at 6.7 TB/s (101 %
// of the measured copy rate).  One token, 8 experts, 7168 -> 2048: 41 us
// (86 %).  One token, NVFP4 8192 x 8192: 14 us against 5.6 us for its bytes:
// launch, first loads and the join of the split rows.
//
// Every wait is bounded (see tc_wait); a CTA that gives up sets its bit in the
// status word, waits for its own copies and leaves.
#pragma once

#include <cuda.h>

#include "farn_product.cuh"
#include "farn_tcgen05.cuh"

namespace farn {

constexpr int kTcMaxStages = 12;
constexpr int kTcMaxSplit = 4;         // CTAs that split a row
constexpr int kTcRowBytes = 128;       // bytes of a row per stage: one swizzle span
constexpr int kTcWeights = 128;        // weights per CTA and tile
// Further warps for gathered rows.  Each takes every sixth stage.  They may
// not be more than the ring has stages: a warp that waits for a stage has to
// be within one round of the ring, or the parity of the phase it waits for
// says nothing.
constexpr int kTcAuxGather = 6;
// NVFP4: block scales come for four stages at a time (64 bytes of a row), in
// blocks of 128 rows (one of weights, the others of slots) that lie in a ring
// of two slots of their own.  Four slots of two stages each cost the matrix
// warp more hand-overs (8192^3: 184 us against 172), three slots of four left
// the ring a stage less (181 against 179).
// Further warps to a block: one if TMA brings it, else (COPY) four, of 32 rows
// each (two of 64 rows took longer for the shifting than the products).
constexpr int kTcScaleStages = 4;
constexpr int kTcScaleSlots = 2;
constexpr int kTcScaleRow = 16 * kTcScaleStages;      // bytes
constexpr int kTcScaleBlock = 128 * kTcScaleRow;
constexpr int kTcCopyWarps = 4;
constexpr int kErrTcFull = 16;         // status bits: matrix warp waiting for operands,
constexpr int kErrTcEmpty = 32;        // producers waiting for a free stage,
constexpr int kErrTcTile = 64;         // epilogue or matrix warp waiting for a tile,
constexpr int kErrTcJoin = 128;        // epilogue waiting for the other parts of the row

struct TcParams {
  ProductParams p;
  int stages;
  int ks;            // CTAs of a cluster that split the row (CG = 1)
  int store_bytes;   // 16, 8 or 2: what N and out allow a store of a row to be
  uint32_t groups_at;  // shared-memory offsets
  uint32_t scales_at;  // NVFP4: the slots of block scales
  uint32_t barriers_at;
  uint32_t part_at;    // fp32 [BN][kPartPitch] for ks > 1, else kTurnBytes for each
                       // epilogue warp
};

struct TcBarriers {
  uint64_t full[kTcMaxStages];
  uint64_t scale_raw[kTcScaleSlots][3];   // a block of scales has landed, as it lies in memory
  uint64_t scale_full[kTcScaleSlots];     // the slot's scales are as the tensor cores read them
  uint64_t scale_empty[kTcScaleSlots];
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
// An epilogue warp's 16 pairs of slots by 32 weights, a word per pair; rows
// of 36 words keep the 16-byte reads free of bank conflicts.
constexpr int kTurnPitch = 36;
constexpr int kTurnBytes = 16 * kTurnPitch * 4;

template <bool FP4, int CG, int BN, bool GATHER, bool COPY>
struct TcShape {
  static constexpr int kSlotBlocks = (BN + 127) / 128;       // blocks of 128 slots' scales
  static constexpr int kScaleWarps = COPY ? kTcCopyWarps : 1;
  static constexpr int kAux = FP4 ? kScaleWarps * (1 + kSlotBlocks) : GATHER ? kTcAuxGather : 0;
  // four epilogue warps, the weights' producer, the matrix warp, and unless
  // the rows are gathered the slots' producer; then the further ones
  static constexpr int kFirstAux = GATHER ? 6 : 7;
  static constexpr int kWarps = kFirstAux + kAux;
  static constexpr int kRows = BN / CG;                      // slots per CTA
  static constexpr int kBox = kRows % 32 == 0 ? 32 : 16;     // rows of a TMA box
  static constexpr int kABytes = kTcWeights * kTcRowBytes;
  static constexpr int kBBytes = kRows * kTcRowBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kScaleSlot = FP4 ? kTcScaleBlock * (1 + kSlotBlocks) : 0;
  static constexpr int kScaleCols = FP4 ? 16 * (1 + kSlotBlocks) : 0;
  static constexpr int kColsUsed = 2 * BN + kScaleCols;
  static constexpr int kCols = kColsUsed <= 128 ? 128 : kColsUsed <= 256 ? 256 : 512;
  static constexpr int kChunk = FP4 ? 256 : 64;              // elements of a row per stage
  static constexpr int kMapStep = FP4 ? kTcRowBytes : kChunk;  // the same in map elements
  static constexpr int kStep = 16 * CG;                      // granularity of a tile's slots
  static_assert(kColsUsed <= 512 && kBBytes % 1024 == 0 && BN % 32 == 0, "");
};

// A tile's slots as one CTA's part of the matrix instruction's N side.
struct SlotRows {
  int first;        // slot
  bool whole;       // one box of all rows, else `loads` boxes of a few
  int loads;
  uint32_t bytes;
};
template <typename Sh, int CG>
__device__ __forceinline__ SlotRows slot_rows(const Tile& w, int w_rank) {
  const int rows = (w.n + Sh::kStep - 1) / Sh::kStep * Sh::kStep / CG;
  SlotRows r;
  r.first = w.slot0 + w_rank * rows;
  r.whole = rows > Sh::kRows - Sh::kBox;
  r.loads = (rows + Sh::kBox - 1) / Sh::kBox;
  r.bytes = (uint32_t)(r.whole ? Sh::kRows : r.loads * Sh::kBox) * kTcRowBytes;
  return r;
}

// Bounded phase wait.  CLUSTER: other CTAs of the cluster arrive on the barrier
// too, so the wait acquires at the cluster's scope.  A waiting thread sleeps:
// nine warps polling took the matrix warp's issue slots (bf16 8192^3 768 us).
constexpr uint32_t kTcSleepNs = 1000000;

template <bool CLUSTER>
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                        int* err, int code) {
  if (tc::mbar_wait_some<CLUSTER>(bar, parity, kTcSleepNs)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (tc::mbar_wait_some<CLUSTER>(bar, parity, kTcSleepNs)) return true;
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

// A value that all lanes hold, in a form that the compiler takes for uniform:
// the matrix instructions' operands then need no move of their own.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// The same by a whole warp, whose lanes go on or give up together.
template <bool CLUSTER>
__device__ __forceinline__ bool tc_wait_warp(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag, int* err, int code) {
  return __all_sync(0xFFFFFFFFu, tc_wait<CLUSTER>(bar, parity, abort_flag, err, code));
}

// Block scales in shared memory, as the tensor cores read them: 128 rows by
// 4 bytes (64 elements) are an atom of 512 bytes, in which row r's four bytes
// are word r / 32 of the 16-byte entry r % 32.  A block of 128 rows by 64
// bytes is 16 atoms, in the order of the row.
//
// A block that TMA wrote as it lies in memory (64-byte rows under the 64-byte
// swizzle, which moves 16-byte piece q of row r to q ^ (r / 2 % 4)), turned
// into atoms in place by one warp: lane l holds the rows l, l + 32, ...
__device__ __forceinline__ void turn_scales(unsigned char* block, int lane) {
  uint4 v[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int row = r * 32 + lane;
      v[r][q] = *reinterpret_cast<const uint4*>(block + row * 64 + ((q ^ ((row >> 1) & 3)) << 4));
    }
  __syncwarp();       // all of it is read before any is written
  uint4* to = reinterpret_cast<uint4*>(block) + lane;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    to[(q * 4 + 0) * 32] = make_uint4(v[0][q].x, v[1][q].x, v[2][q].x, v[3][q].x);
    to[(q * 4 + 1) * 32] = make_uint4(v[0][q].y, v[1][q].y, v[2][q].y, v[3][q].y);
    to[(q * 4 + 2) * 32] = make_uint4(v[0][q].z, v[1][q].z, v[2][q].z, v[3][q].z);
    to[(q * 4 + 3) * 32] = make_uint4(v[0][q].w, v[1][q].w, v[2][q].w, v[3][q].w);
  }
}

// 16 bytes at `at`, a multiple of 16, of which those outside [lo, hi) are not
// read.
static __device__ __noinline__ uint4 load_within(uintptr_t at, uintptr_t lo, uintptr_t hi) {
  if (at >= lo && at + 16 <= hi) return __ldg(reinterpret_cast<const uint4*>(at));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (at + i >= lo && at + i < hi)
      w[i >> 2] |= (uint32_t)__ldg(reinterpret_cast<const uint8_t*>(at + i)) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 32 rows of a block whose rows in memory start at any byte (H not a multiple
// of 256), by one warp: five lanes read the five aligned 16-byte pieces that
// 64 bytes can touch, six rows to a load and all six loads in flight; the
// words are then shifted into place with the next lane's first.
struct ScaleRows {
  const uint8_t* src;    // the first of the rows
  int rows;              // rows that exist (32 at most); the others are 0
  int left;              // bytes of a row from src on; what follows is 0
};
constexpr int kScalePieces = 5;
constexpr int kScaleRows = 6;        // per load
constexpr int kScaleLoads = 6;

// [lo, hi): the whole tensor, outside of which nothing is read.
__device__ __forceinline__ void load_scale_rows(uint4* v, const ScaleRows& b, int64_t pitch,
                                                uintptr_t lo, uintptr_t hi, int lane) {
  const int piece = lane % kScalePieces, sub = lane / kScalePieces;
  const int lim = b.left < kTcScaleRow ? b.left : kTcScaleRow;
  const uintptr_t first = (uintptr_t)b.src;
  // only the tensor's first and last rows have pieces that reach out of it
  const bool inside = (first & ~(uintptr_t)15) >= lo &&
                      first + (b.rows - 1) * pitch + lim + 15 <= hi;
  if (inside) {
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
      const int k = i * kScaleRows + sub;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      const uintptr_t a = first + k * pitch, at = (a & ~(uintptr_t)15) + piece * 16;
      if (sub < kScaleRows && k < b.rows && at < a + lim)
        v[i] = __ldg(reinterpret_cast<const uint4*>(at));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
      const int k = i * kScaleRows + sub;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      const uintptr_t a = first + k * pitch, at = (a & ~(uintptr_t)15) + piece * 16;
      if (sub < kScaleRows && k < b.rows && at < a + lim) v[i] = load_within(at, lo, hi);
    }
  }
}

// quarter: the rows' place in the block, which is one word of every entry
__device__ __forceinline__ void put_scale_rows(unsigned char* block, const uint4* v,
                                               const ScaleRows& b, int64_t pitch,
                                               int quarter, int lane) {
  const int piece = lane % kScalePieces, sub = lane / kScalePieces;
  const int lim = b.left < kTcScaleRow ? b.left : kTcScaleRow;
  const uint32_t low = (uint32_t)(uintptr_t)b.src, step = (uint32_t)pitch;
#pragma unroll
  for (int i = 0; i < kScaleLoads; ++i) {
    const int k = i * kScaleRows + sub;
    const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, v[i].x, 1);
    const uint32_t off = (low + k * step) & 15u, by = 8 * (off & 3u);
    const uint32_t w[5] = {v[i].x, v[i].y, v[i].z, v[i].w, next};
    const int b0 = piece * 16 - (int)(off & 12u);
    const int to = k * 16 + quarter * 4 + b0 * 128;
    const bool mine = sub < kScaleRows && k < 32;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = b0 + 4 * j;
      uint32_t word = __funnelshift_r(w[j], w[j + 1], by);
      if (lim < kTcScaleRow && at + 4 > lim)
        word = at >= lim ? 0u : word & ((1u << (8 * (lim - at))) - 1u);
      if (mine && (uint32_t)at < (uint32_t)kTcScaleRow)
        *reinterpret_cast<uint32_t*>(block + to + 512 * j) = word;
    }
  }
}

// Up to 32 slots by the warp's 32 weights, from the accumulator's columns at
// `tmem` to rows of the output.  The accumulator has a weight per lane; the
// warp turns it over in shared memory, two slots to a word, and writes runs
// of eight weights if rows are so aligned (about 110 instructions for 1024 values; one warp per
// scheduler issues one in 4 to 5 cycles, so their number is the time).
// v[j]: slot j's product with the lane's weight; n: slots; live: those whose
// row exists; first: the warp's first weight; store_bytes: 16, 8 or 2, what N
// and out allow a store of a row to be.
template <bool GATHER>
__device__ __forceinline__ void store_columns(const ProductParams& p, int store_bytes,
                                              const uint32_t* v, uint32_t* turn, int64_t slot,
                                              int n, uint32_t live, int64_t first, int lane) {
  const float alpha = p.alpha;
  if (store_bytes == 2) {
    // Rows that start anywhere: straight from the registers, a store being one
    // slot's run of the warp's 32 weights (in runs of eight, element by
    // element, such an N took twice the time; turned and in words 16 % more).
    const int64_t w = first + lane;
    uint16_t* o = static_cast<uint16_t*>(p.out) + slot * p.N + w;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j < n && w < p.N)
        *o = GATHER && !((live >> j) & 1u) ? (uint16_t)0 : to_bf16(__uint_as_float(v[j]) * alpha);
      o += p.N;
      asm volatile("" : "+l"(o));     // one address at a time, not 32 in registers
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j)
    turn[j * kTurnPitch + lane] = pack_bf16x2(__uint_as_float(v[2 * j]) * alpha,
                                              __uint_as_float(v[2 * j + 1]) * alpha);
  __syncwarp();
  const int oct = lane & 3;
  const int64_t col = first + oct * 8;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int pair = h * 8 + (lane >> 2);
    const uint4 a = *reinterpret_cast<const uint4*>(turn + pair * kTurnPitch + oct * 8);
    const uint4 b = *reinterpret_cast<const uint4*>(turn + pair * kTurnPitch + oct * 8 + 4);
    uint4 w[2];
    w[0] = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                      __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
    w[1] = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                      __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = pair * 2 + i;
      if (s >= n || col >= p.N) continue;
      if (GATHER && !((live >> s) & 1u)) w[i] = make_uint4(0u, 0u, 0u, 0u);
      uint16_t* o = static_cast<uint16_t*>(p.out) + (slot + s) * p.N + col;
      if (store_bytes == 16) {
        *reinterpret_cast<uint4*>(o) = w[i];
      } else {
        *reinterpret_cast<uint2*>(o) = make_uint2(w[i].x, w[i].y);
        if (col + 4 < p.N) reinterpret_cast<uint2*>(o)[1] = make_uint2(w[i].z, w[i].w);
      }
    }
  }
  __syncwarp();
}
template <bool GATHER>
__device__ __forceinline__ void store_turned(const TcParams& t, uint32_t tmem, uint32_t* turn,
                                             int64_t slot, int n, uint32_t live, int64_t first,
                                             int lane) {
  uint32_t v[32];
  tc::tmem_ld32(tmem, v);
  tc::tmem_ld_wait();
  store_columns<GATHER>(t.p, t.store_bytes, v, turn, slot, n, live, first, lane);
}

template <bool FP4, int CG, int BN, bool GATHER, bool COPY>
__global__ void __launch_bounds__(TcShape<FP4, CG, BN, GATHER, COPY>::kWarps * 32, 1)
farn_product_tc_kernel(const __grid_constant__ TcParams t,
                       const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ CUtensorMap map_x,
                       const __grid_constant__ CUtensorMap map_part,
                       const __grid_constant__ CUtensorMap map_ws,
                       const __grid_constant__ CUtensorMap map_xs) {
  using Sh = TcShape<FP4, CG, BN, GATHER, COPY>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const ProductParams& p = t.p;
  const uint32_t base = (tc::smem_addr(smem_raw) + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - tc::smem_addr(smem_raw));
  const uint32_t NS = t.stages;
  TcBarriers* bb = reinterpret_cast<TcBarriers*>(smem + t.barriers_at);
  const Groups g = groups_at(smem + t.groups_at, p.E);
  const uint32_t full0 = tc::smem_addr(&bb->full[0]);
  const uint32_t empty0 = tc::smem_addr(&bb->empty[0]);
  const uint32_t sraw0 = tc::smem_addr(&bb->scale_raw[0][0]);
  const uint32_t sfull0 = tc::smem_addr(&bb->scale_full[0]);
  const uint32_t sempty0 = tc::smem_addr(&bb->scale_empty[0]);
  const uint32_t tfull0 = tc::smem_addr(&bb->tile_full[0]);
  const uint32_t tempty0 = tc::smem_addr(&bb->tile_empty[0]);
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
    if (lane < 2) {
      mbar_init(tfull0 + 8 * lane, 1);
      mbar_init(tempty0 + 8 * lane, 4 * CG);
    }
    if (FP4 && lane < kTcScaleSlots) {
      mbar_init(sfull0 + 8 * lane, Sh::kScaleWarps * (1 + Sh::kSlotBlocks) * CG);
      mbar_init(sempty0 + 8 * lane, 1);
      for (int u = 0; u < 3; ++u) mbar_init(sraw0 + 8 * (lane * 3 + u), 1);
    }
    if (lane == 0) {
      mbar_init(tc::smem_addr(&bb->part_full), 4 * csize);
      mbar_init(tc::smem_addr(&bb->part_empty), 4 * csize);
      mbar_init(tc::smem_addr(&bb->never), 1);
      bb->abort_flag = 0;
    }
    tc::mbar_init_fence();
  }
  if (warp == 5) tc::tmem_alloc<CG>(tc::smem_addr(&bb->tmem), Sh::kCols);
  if (tid == 4 * 32) {
    tc::prefetch_map(&map_w);
    if constexpr (!GATHER) {
      tc::prefetch_map(&map_x);
      tc::prefetch_map(&map_part);
    }
    if (FP4 && !COPY) {
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
  const uint32_t tmem = uniform(bb->tmem);

  constexpr int kTileWeights = kTcWeights * CG;
  constexpr bool kPair = CG == 2;   // the other CTA arrives on a tile's barriers too
  const int wts = (int)((p.N + kTileWeights - 1) / kTileWeights);
  const int32_t tiles = g.tile[p.E] * wts;
  const int32_t t0 = blockIdx.x / csize, tstep = gridDim.x / csize;
  const int chunks = (int)((p.H + Sh::kChunk - 1) / Sh::kChunk);
  const int c0 = CG == 2 ? 0 : (int)((int64_t)chunks * rank / csize);
  const int c1 = CG == 2 ? chunks : (int)((int64_t)chunks * (rank + 1) / csize);
  const int nc = c1 - c0;
  const int w_rank = CG == 2 ? (int)rank : 0;      // this CTA's part of a tile's weights

  if (warp == 4) {
    // ------------------------------------------------- weights' producer
    const uint32_t bar0 = tc::map_rank(full0, CG == 2 ? 0 : rank);
    RingPos at;
    uint32_t armed = 0;        // stages given to TMA, all but the last NS done
    bool ok = true;
    if (t.p.stall_test && blockIdx.x == 0)
      ok = tc_wait_warp<false>(tc::smem_addr(&bb->never), 0, abort_flag, p.err, kErrTcEmpty);
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      const SlotRows r = slot_rows<Sh, CG>(w, w_rank);
      const uint32_t bytes = CG * (Sh::kABytes + (GATHER ? 0 : r.bytes));
      const int n0 = w.wt * kTileWeights + w_rank * kTcWeights;
      for (int c = c0; c < c1; ++c, at.next(NS), ++armed) {
        const uint32_t s = at.stage;
        ok = tc_wait_warp<kPair>(empty0 + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        if (tc::elect_one()) {
          if (w_rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, bytes);
          tc::load_3d<CG>(base + s * Sh::kStageBytes, &map_w, c * Sh::kMapStep, n0, w.e,
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
  } else if (warp == 5) {
    // ------------------------------------------------- matrix instructions
    if (w_rank == 0) {
      RingPos at;
      uint32_t nt = 0;
      bool ok = true;
      const uint64_t desc0 = tc::operand_desc(base);
      const uint64_t scale0 = tc::scale_desc(base + t.scales_at);
      uint32_t ng = 0;           // groups of scales so far
      const uint32_t sf_a = tmem + 2 * BN, sf_b = sf_a + 16;
      for (int32_t tile = t0; ok && tile < tiles; tile += tstep, ++nt) {
        const Tile w = find_tile(g, p.E, tile, wts, BN);
        const int n_eff = (w.n + Sh::kStep - 1) / Sh::kStep * Sh::kStep;
        const uint32_t idesc = FP4 ? tc::idesc_nvfp4(kTileWeights, n_eff)
                                   : tc::idesc_bf16(kTileWeights, n_eff);
        const uint32_t acc = nt & 1, d = tmem + acc * BN;
        ok = tc_wait_warp<kPair>(tempty0 + 8 * acc, ((nt >> 1) & 1) ^ 1, abort_flag, p.err,
                                 kErrTcTile);
        if (!ok) break;
        tc::fence_after();
        // Few instructions per stage: a dependent one costs this warp about
        // ten cycles, and a stage's NVFP4 products take 450.
        uint32_t more = 0;                 // 0 before the tile's first product
        for (int c = 0; ok && c < nc;) {
          uint64_t sc = 0;
          int end = nc;
          if constexpr (FP4) {
            const uint32_t slot = ng % kTcScaleSlots;
            ok = tc_wait_warp<kPair>(sfull0 + 8 * slot, ng / kTcScaleSlots & 1, abort_flag, p.err,
                                     kErrTcFull);
            sc = scale0 + (slot * Sh::kScaleSlot >> 4);
            end = min(nc, c + kTcScaleStages);
          }
          for (; ok && c < end; ++c) {
            const uint32_t s = at.stage;
            ok = tc_wait_warp<kPair>(full0 + 8 * s, at.phase, abort_flag, p.err, kErrTcFull);
            if (!ok) break;
            tc::fence_after();
            const uint64_t da = desc0 + (s * Sh::kStageBytes >> 4), db = da + (Sh::kABytes >> 4);
            if (tc::elect_one()) {
              if constexpr (FP4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  tc::copy_scales<CG>(sf_a + 4 * k, sc + (512 >> 4) * k);
#pragma unroll
                  for (int j = 0; j < Sh::kSlotBlocks; ++j)
                    if (j == 0 || n_eff > 128)
                      tc::copy_scales<CG>(sf_b + (k * Sh::kSlotBlocks + j) * 4,
                                          sc + (kTcScaleBlock >> 4) * (1 + j) + (512 >> 4) * k);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  tc::mma_nvfp4<CG>(d, da + 2 * k, db + 2 * k, idesc, sf_a + 4 * k,
                                    sf_b + 4 * k * Sh::kSlotBlocks, k > 0 ? 1u : more);
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  tc::mma_bf16<CG>(d, da + 2 * k, db + 2 * k, idesc, k > 0 ? 1u : more);
              }
              tc::commit<CG>(empty0 + 8 * s);
            }
            more = 1;
            sc += 2048 >> 4;
            at.next(NS);
          }
          if (!ok) break;
          if (tc::elect_one()) {
            if constexpr (FP4) tc::commit<CG>(sempty0 + 8 * (ng % kTcScaleSlots));
            if (c == nc) tc::commit<CG>(tfull0 + 8 * acc);
          }
          ++ng;
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
    uint32_t* turn = reinterpret_cast<uint32_t*>(smem + t.part_at + warp * kTurnBytes);
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep, ++nt) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      const uint32_t acc = nt & 1, d = tmem + acc * BN + ((uint32_t)warp << 21);
      const int64_t n0 = (int64_t)w.wt * kTileWeights + w_rank * kTcWeights;
      ok = tc_wait_warp<kPair>(tfull0 + 8 * acc, (nt >> 1) & 1, abort_flag, p.err, kErrTcTile);
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
        for (int c = 0; c < w.n; c += 32) {
          uint32_t live = 0xFFFFFFFFu;
          if constexpr (GATHER) {
            const int r = c + lane < w.n ? p.rows[(int64_t)w.slot0 + c + lane] : -1;
            live = __ballot_sync(0xFFFFFFFFu, r >= 0 && r < p.n_a);
          }
          store_turned<GATHER>(t, d + c, turn, (int64_t)w.slot0 + c, w.n - c, live,
                               n0 + warp * 32, lane);
        }
      }
      tc::fence_before();       // orders the reads of tensor memory before the arrival
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_first<CG>(tempty0 + 8 * acc);
      if (split) {
        if (lane < csize) tc::mbar_arrive_cluster(tc::map_rank(part_full, lane));
        ok = tc_wait_warp<true>(part_full, nt & 1, abort_flag, p.err, kErrTcJoin);
        if (!ok) break;
        // each CTA sums its share of the tile, four weights to a thread, the
        // parts in rank order; two quads' loads are in flight together
        const uint32_t mine = tc::smem_addr(part);
        const int quads = w.n * (kTcWeights / 4), step = csize * 128;
        for (int i0 = (int)rank * 128 + tid; i0 < quads; i0 += 2 * step) {
          float4 v[2][kTcMaxSplit];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int i = i0 + h * step;
            const uint32_t at = ((i >> 5) * kPartPitch + (i & 31) * 4) * 4;
#pragma unroll
            for (int q = 0; q < kTcMaxSplit; ++q)
              if (q < csize && i < quads) v[h][q] = tc::ld_cluster_v4(tc::map_rank(mine, q) + at);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int i = i0 + h * step;
            if (i >= quads) break;
            float4 sum = v[h][0];
#pragma unroll
            for (int q = 1; q < kTcMaxSplit; ++q)
              if (q < csize) {
                sum.x += v[h][q].x; sum.y += v[h][q].y; sum.z += v[h][q].z; sum.w += v[h][q].w;
              }
            const int64_t s = (int64_t)w.slot0 + (i >> 5), n = n0 + (i & 31) * 4;
            if constexpr (GATHER)
              if (p.rows[s] < 0 || p.rows[s] >= p.n_a) sum = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t e[2] = {pack_bf16x2(sum.x * p.alpha, sum.y * p.alpha),
                                   pack_bf16x2(sum.z * p.alpha, sum.w * p.alpha)};
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
        }
        __syncwarp();
        if (lane < csize) tc::mbar_arrive_cluster(tc::map_rank(part_empty, lane));
      }
    }
  } else if (!GATHER && warp == 6) {
    // --------------------------------------------------- slots' producer
    const uint32_t bar0 = tc::map_rank(full0, CG == 2 ? 0 : rank);
    RingPos at;
    bool ok = true;
    for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
      const Tile w = find_tile(g, p.E, tile, wts, BN);
      const SlotRows r = slot_rows<Sh, CG>(w, w_rank);
      for (int c = c0; c < c1; ++c, at.next(NS)) {
        const uint32_t s = at.stage;
        ok = tc_wait_warp<kPair>(empty0 + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
        if (!ok) break;
        const uint32_t b = base + s * Sh::kStageBytes + Sh::kABytes;
        if (tc::elect_one()) {
          if (r.whole) {
            tc::load_2d<CG>(b, &map_x, c * Sh::kMapStep, r.first, bar0 + 8 * s);
          } else {
            for (int i = 0; i < r.loads; ++i)
              tc::load_2d<CG>(b + i * Sh::kBox * kTcRowBytes, &map_part, c * Sh::kMapStep,
                              r.first + i * Sh::kBox, bar0 + 8 * s);
          }
        }
        __syncwarp();
      }
    }
  } else if constexpr (FP4) {
    // ------------------------------------------------------- block scales
    const int u = (warp - Sh::kFirstAux) / Sh::kScaleWarps;             // block
    const int quarter = (warp - Sh::kFirstAux) % Sh::kScaleWarps;       // its warp
    const int64_t pitch = p.H / 16;
    const int groups = (nc + kTcScaleStages - 1) / kTcScaleStages;
    unsigned char* block0 = smem + t.scales_at + u * kTcScaleBlock;
    bool ok = true;
    if constexpr (!COPY) {
      // TMA brings a block as it lies and one warp turns it; the next group's
      // copy is on its way while this one's products run.  Both CTAs of a
      // pair need all slots' scales, and each loads them for itself.
      int32_t tile = t0;
      int gi = 0;                             // group of the tile
      uint32_t asked = 0, done = 0;           // groups so far
      uint32_t coming = 0;                    // slots whose block TMA was asked for, a bit each
      Tile w = {};
      auto ask = [&]() {                      // false: no more, or gave up
        if (tile >= tiles) return false;
        if (gi == 0) w = find_tile(g, p.E, tile, wts, BN);
        const uint32_t slot = asked % kTcScaleSlots;
        if (!tc_wait_warp<kPair>(sempty0 + 8 * slot, (asked / kTcScaleSlots & 1) ^ 1, abort_flag,
                                 p.err, kErrTcEmpty)) {
          ok = false;
          return false;
        }
        // slots above 128 that the tile does not have are not loaded
        coming &= ~(1u << slot);
        if (u < 2 || w.n > 128) {
          coming |= 1u << slot;
          if (tc::elect_one()) {
            const uint32_t bar = sraw0 + 8 * (slot * 3 + u);
            const uint32_t dst = base + t.scales_at + slot * Sh::kScaleSlot + u * kTcScaleBlock;
            const int x = (c0 + gi * kTcScaleStages) * 16;
            mbar_arrive_expect_tx(bar, kTcScaleBlock);
            if (u == 0)
              tc::load_2d<1>(dst, &map_ws, x, w.wt * kTileWeights + w_rank * kTcWeights, bar);
            else
              tc::load_2d<1>(dst, &map_xs, x, w.slot0 + (u - 1) * 128, bar);
          }
          __syncwarp();
        }
        ++asked;
        if (++gi == groups) { gi = 0; tile += tstep; }
        return true;
      };
      {
        uint32_t phases = 0;        // of each slot's raw barrier, a bit each
        bool more = true;
        for (int i = 0; more && i < kTcScaleSlots; ++i) more = ask();
        for (int32_t at = t0; ok && at < tiles; at += tstep) {
          const int n = find_tile(g, p.E, at, wts, BN).n;
          for (int i = 0; ok && i < groups; ++i, ++done) {
            const uint32_t slot = done % kTcScaleSlots;
            if (u < 2 || n > 128) {
              ok = tc_wait_warp<false>(sraw0 + 8 * (slot * 3 + u), phases >> slot & 1, abort_flag,
                                       p.err, kErrTcFull);
              if (!ok) break;
              phases ^= 1u << slot;
              turn_scales(block0 + slot * Sh::kScaleSlot, lane);
              tc::fence_async_shared();
            }
            __syncwarp();
            if (lane == 0)
              tc::mbar_arrive_first<CG>(sfull0 + 8 * slot);
            // the last slot is the one of the group before this, when its
            // products are done; this one is turned by then
            if (more && done > 0) more = ask();
          }
        }
        // after an abort: what was asked for lands before the CTA leaves
        for (; done < asked; ++done) {
          const uint32_t slot = done % kTcScaleSlots;
          if (!(coming >> slot & 1)) continue;
          const uint64_t begin = globaltimer_ns();
          while (!tc::mbar_wait_some<true>(sraw0 + 8 * (slot * 3 + u), phases >> slot & 1,
                                           kTcSleepNs) &&
                 globaltimer_ns() - begin < kWaitLimitNs) {}
          phases ^= 1u << slot;
        }
      }
    } else {
      const uintptr_t lo = (uintptr_t)(u ? p.a_scale : p.b_scale);
      const uintptr_t hi = lo + (u ? p.n_a : p.N) * pitch;
      // The next group's rows are on their way while the warp waits for a
      // slot.
      int32_t tile = t0;
      int gi = 0;
      Tile w = {};
      auto next = [&]() {
        if (gi == 0) w = find_tile(g, p.E, tile, wts, BN);
        const int64_t n0 = (int64_t)w.wt * kTileWeights + w_rank * kTcWeights;
        const int first = (u ? (u - 1) * 128 : 0) + quarter * 32;
        const int64_t x = (int64_t)(c0 + gi * kTcScaleStages) * 16;
        ScaleRows b;
        b.src = (u ? p.a_scale + ((int64_t)w.slot0 + first) * pitch
                   : p.b_scale + (n0 + first) * pitch) + x;
        b.rows = (int)min((u ? (int64_t)w.n : p.N - n0) - first, (int64_t)32);
        b.left = (int)min(pitch - x, (int64_t)kTcScaleRow);
        if (++gi == groups) { gi = 0; tile += tstep; }
        return b;
      };
      uint4 v[kScaleLoads];
      ScaleRows b = {};
      bool more = tile < tiles;
      if (more) {
        b = next();
        load_scale_rows(v, b, pitch, lo, hi, lane);
      }
      for (uint32_t ng = 0; more; ++ng) {
        const uint32_t slot = ng % kTcScaleSlots;
        ok = tc_wait_warp<kPair>(sempty0 + 8 * slot, (ng / kTcScaleSlots & 1) ^ 1, abort_flag,
                                 p.err, kErrTcEmpty);
        if (!ok) break;
        put_scale_rows(block0 + slot * Sh::kScaleSlot, v, b, pitch, quarter, lane);
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0)
          tc::mbar_arrive_first<CG>(sfull0 + 8 * slot);
        more = tile < tiles;
        if (more) {           // after the fence, which waits for loads too
          b = next();
          load_scale_rows(v, b, pitch, lo, hi, lane);
        }
      }
    }
  }

  if constexpr (GATHER) {
    if (warp >= Sh::kFirstAux) {
      // ------------------------------------------------------ gathered rows
      // A warp takes every sixth stage, so that a stage's copies have the whole
      // ring's time to land.  Eight lanes copy a row's 128 bytes, in the
      // swizzled layout that TMA would write: 16-byte column j of row r at
      // j ^ (r & 7).  Lane l knows the rows l, l + 32, l + 64 and l + 96.
      constexpr int kHeld = (Sh::kRows + 31) / 32;
      const int mine = warp - Sh::kFirstAux, col = lane & 7, sub = lane >> 3;
      const char* x = static_cast<const char*>(p.a) + col * 16;
      const uint64_t pitch = (uint64_t)p.H * 2;
      RingPos at;
      at.skip(mine, NS);
      int ahead = mine;
      bool ok = true;
      for (int32_t tile = t0; ok && tile < tiles; tile += tstep) {
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
          ok = tc_wait_warp<kPair>(empty0 + 8 * s, at.phase ^ 1, abort_flag, p.err, kErrTcEmpty);
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
            tc::mbar_arrive_first<CG>(full0 + 8 * s);
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

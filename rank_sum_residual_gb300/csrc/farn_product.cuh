// The products' parameters, the walk over their tiles, and the kernel that
// takes every shape.
//
// Both products have one form: out[s, n] = alpha * sum_h a[s, h] * b_e[n, h]
// for the slots s of group e.  The dense NVFP4 product is one group.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "farn_kernels.cuh"

namespace farn {

constexpr int kMaxExperts = 1024;

struct ProductParams {
  const void* a;          // bf16 [n_a, H], or NVFP4 codes [S, H / 2]
  const uint8_t* a_scale; // NVFP4: [S, H / 16]
  const void* b;          // bf16 [E, N, H], or NVFP4 codes [N, H / 2]
  const uint8_t* b_scale; // NVFP4: [N, H / 16]
  const int32_t* rows;    // [S] the row of a that slot s reads, or null: row s
  const int32_t* offsets; // [E + 1], or null: one group of S slots
  void* out;              // bf16 [S, N]
  int64_t n_a, S, N, H;
  int E;
  float alpha;
  int* err;               // device status word
  int stall_test;         // a test of the bounded waits (see farn_create)
};

// The groups' slots and tiles, in shared memory: first[e] .. first[e] +
// count[e] - 1 are the slots of group e, tile[e] the number of slot tiles
// before it.  Offsets are clamped to 0..S and to what came before them, so
// that the groups are disjoint and no value of them leads outside the tensors.
struct Groups {
  int32_t* first;   // [E]
  int32_t* count;   // [E]
  int32_t* tile;    // [E + 1]
};
__host__ __device__ constexpr uint32_t groups_bytes(int E) { return (3u * E + 1u) * 4u; }
__device__ __forceinline__ Groups groups_at(void* smem, int E) {
  int32_t* v = static_cast<int32_t*>(smem);
  return Groups{v, v + E, v + 2 * E};
}

// By all threads of the block (a multiple of 32, at least 64).
__device__ __forceinline__ void load_groups(const Groups& g, const ProductParams& p, int bn) {
  const int tid = threadIdx.x, lane = tid & 31;
  // the end of every group first: the loads of all are in flight together
  for (int e = tid; e < p.E; e += blockDim.x)
    g.count[e] = (int32_t)(p.offsets ? min(max((int64_t)p.offsets[e + 1], (int64_t)0), p.S) : p.S);
  int32_t end =
      (int32_t)(p.offsets ? min(max((int64_t)p.offsets[0], (int64_t)0), p.S) : (int64_t)0);
  __syncthreads();
  if (tid < 32) {   // a warp scans the ends (their maximum) and the tiles, 32 groups at a time
    int32_t tiles = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int32_t hi = max(end, e < p.E ? g.count[e] : 0);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, hi, o);
        if (lane >= o) hi = max(hi, y);
      }
      int32_t lo = __shfl_up_sync(0xFFFFFFFFu, hi, 1);
      if (lane == 0) lo = end;
      const int32_t n = e < p.E ? (int32_t)(((int64_t)hi - lo + bn - 1) / bn) : 0;
      int32_t inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
      }
      if (e < p.E) {
        g.first[e] = lo;
        g.count[e] = hi - lo;
        g.tile[e] = tiles + inc - n;
      }
      end = __shfl_sync(0xFFFFFFFFu, hi, 31);
      tiles += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    if (lane == 0) g.tile[p.E] = tiles;
  }
  __syncthreads();
}

struct Tile {
  int e;
  int32_t slot0;   // first slot
  int n;           // slots (1 .. bn)
  int wt;          // weight tile
};

// Tile t (the host keeps their number below 2^31) of the walk over all groups,
// by a whole warp; wts: weight tiles per
// group.  Within a
// group the walk covers kSuper slot tiles by all weight tiles before it goes
// on, slot tiles fastest, so that the tiles in flight at a time share both
// operands' rows in L2.
constexpr int kSuper = 8;

__device__ __forceinline__ Tile find_tile(const Groups& g, int E, int32_t t, int wts, int bn) {
  const int32_t q = t / wts;
  int lo = 0, hi = E - 1;            // the last e with tile[e] <= q
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.tile[mid] <= q) lo = mid; else hi = mid - 1;
  }
  const int32_t st = g.tile[lo + 1] - g.tile[lo];       // slot tiles of the group
  const int32_t local = t - g.tile[lo] * wts;
  const int32_t per = kSuper * wts;
  const int32_t sup = local / per;
  const int32_t in = local - sup * per;
  const int32_t width = min(kSuper, st - sup * kSuper);
  // The group's tiles are of one size (a multiple of 32, or of bn below
  // that), rather than full ones and a rest: a tile of few slots streams its
  // weights for little work.  None is empty: count > (st - 1) * bn.
  const int32_t count = g.count[lo], step = min(bn, 32);
  const int32_t size = ((count - 1) / st / step + 1) * step;
  Tile r;
  r.e = lo;
  r.wt = in / width;
  const int32_t s = sup * kSuper + (in - r.wt * width);
  r.slot0 = g.first[lo] + s * size;
  r.n = min(size, count - s * size);
  // all lanes hold the same; a broadcast lets the compiler know it, and the
  // TMA and matrix instructions' operands then need no move of their own
  r.e = __shfl_sync(0xFFFFFFFFu, r.e, 0);
  r.wt = __shfl_sync(0xFFFFFFFFu, r.wt, 0);
  r.slot0 = __shfl_sync(0xFFFFFFFFu, r.slot0, 0);
  r.n = __shfl_sync(0xFFFFFFFFu, r.n, 0);
  return r;
}

// ------------------------------------------------------------ any shape
// 64 x 64 outputs per block in fp32 on the CUDA cores, for rows that TMA
// cannot read (H or an address off 16 bytes).  Bound by the fp32 pipe; no
// call with aligned rows takes it.
constexpr int kPlainTile = 64;
constexpr int kPlainK = 16;
constexpr int kPlainThreads = 256;

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, f = c & 1u;
  const float v = e ? __uint_as_float(((e + 126u) << 23) | (f << 22)) : 0.5f * (float)f;
  return (c & 8u) ? -v : v;
}

template <bool FP4>
__device__ __forceinline__ float product_value(const void* t, const uint8_t* scale, int64_t row,
                                               int64_t H, int64_t h) {
  if constexpr (FP4) {
    const uint32_t b = static_cast<const uint8_t*>(t)[(row * H + h) >> 1];
    return e2m1_value((h & 1) ? b >> 4 : b & 15u) *
           e4m3_to_f32(scale[(row * H + h) >> 4]);
  } else {
    return bf_lo((uint32_t) static_cast<const uint16_t*>(t)[row * H + h]);
  }
}

template <bool FP4>
__global__ void __launch_bounds__(kPlainThreads)
farn_product_plain_kernel(const ProductParams p) {
  __shared__ int32_t gmem[groups_bytes(kMaxExperts) / 4];
  const Groups g = groups_at(gmem, p.E);
  __shared__ float as[kPlainK][kPlainTile + 1], bs[kPlainK][kPlainTile + 1];
  pdl_wait();
  pdl_trigger();
  load_groups(g, p, kPlainTile);
  const int tid = threadIdx.x, ti = tid / 16, tj = tid % 16;
  const int wts = (int)((p.N + kPlainTile - 1) / kPlainTile);
  const int32_t tiles = g.tile[p.E] * wts;
  for (int32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const Tile w = find_tile(g, p.E, t, wts, kPlainTile);
    const int64_t n0 = (int64_t)w.wt * kPlainTile;
    float acc[4][4] = {};
    for (int64_t h0 = 0; h0 < p.H; h0 += kPlainK) {
      for (int i = tid; i < kPlainTile * kPlainK; i += kPlainThreads) {
        const int r = i / kPlainK, k = i % kPlainK;
        const int64_t h = h0 + k;
        float va = 0.0f, vb = 0.0f;
        if (h < p.H && r < w.n) {
          const int64_t row = p.rows ? p.rows[w.slot0 + r] : (int64_t)w.slot0 + r;
          if (row >= 0 && row < p.n_a) va = product_value<FP4>(p.a, p.a_scale, row, p.H, h);
        }
        if (h < p.H && n0 + r < p.N)
          vb = product_value<FP4>(p.b, p.b_scale, (int64_t)w.e * p.N + n0 + r, p.H, h);
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
            acc[i][j] = fmaf(as[k][ti * 4 + i], bs[k][tj + 16 * j], acc[i][j]);
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
      const int r = ti * 4 + i;
      if (r >= w.n) break;
      // a slot whose row does not exist has products with zeros; it stays
      // zero whatever the weights hold
      bool live = true;
      if (p.rows) {
        const int64_t row = p.rows[w.slot0 + r];
        live = row >= 0 && row < p.n_a;
      }
      for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + tj + 16 * j;
        if (n < p.N)
          static_cast<uint16_t*>(p.out)[((int64_t)w.slot0 + r) * p.N + n] =
              live ? to_bf16(acc[i][j] * p.alpha) : (uint16_t)0;
      }
    }
  }
}

}  // namespace farn

// The MoE router: top-K experts of every token, their softmax gates, and
// the slots of the (token, expert) pairs sorted by expert.
//
// A block takes a run of tokens, one warp per token at a time.  The K
// experts are found one after the other by a warp-wide maximum over
// order-preserving integers.  The sort by expert needs no atomics whose
// order matters: a block keeps, for every expert, a bit mask of its own
// tokens that chose it, so a pair's place among the block's pairs of the
// same expert is the number of lower bits set, and the block's count is the
// number of bits.  What is left is a scan of the blocks' counts: through
// distributed shared memory where one cluster holds all tokens, else with
// two more kernels.
#include <cooperative_groups.h>
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

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxE = FARN_MAX_EXPERTS;
constexpr int kScanThreads = 1024;
constexpr int kScanCtas = 8;              // cluster of the scan kernel
constexpr int kScanE = kMaxE / kScanCtas; // most experts per CTA of the scan

struct RouteParams {
  const void* logits;
  int64_t T;
  int E, K;
  int renorm;
  int tb;             // tokens per block (a multiple of 32); the last one may have fewer
  int nb;             // blocks
  int32_t* experts;   // [T, K]
  float* gates;       // [T, K]
  int32_t* index;     // [T, K]
  int32_t* rows;      // [T * K]
  int32_t* offsets;   // [E + 1]
};

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* logits, int64_t i) {
  if constexpr (BF16)
    return farn::bf_lo((uint32_t) static_cast<const uint16_t*>(logits)[i]);
  else
    return static_cast<const float*>(logits)[i];
}

// An integer that orders as the value does (-0 and +0 alike); 0 for what is
// never chosen: -inf and NaN.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return v > -INFINITY ? k : 0u;
}
// The value of a non-zero key.
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// exp(v - m) of the value of a non-zero key, 1 where both are the same
// infinity.
__device__ __forceinline__ float weight_of(uint32_t key, float m) {
  const float v = key_value(key);
  return v == m ? 1.0f : expf(v - m);
}

// A candidate as one number that orders by the logit's key, then by the lower
// expert: 16 and 16 bits for bf16 logits, 32 and 32 for fp32 ones.  0: none.
template <bool BF16>
struct Candidate;
template <>
struct Candidate<true> {
  typedef uint32_t Word;
  static __device__ __forceinline__ Word make(uint32_t key, int e) {
    return key ? (key & 0xFFFF0000u) | (0xFFFFu - (uint32_t)e) : 0u;
  }
  // of a bf16 value's key the low half is all ones below zero, else zeros
  static __device__ __forceinline__ uint32_t key(Word w) {
    return (w & 0x80000000u) ? w & 0xFFFF0000u : w | 0xFFFFu;
  }
  static __device__ __forceinline__ int expert(Word w) { return 0xFFFF - (int)(w & 0xFFFFu); }
  static __device__ __forceinline__ Word warp_max(Word w) {
    return __reduce_max_sync(0xFFFFFFFFu, w);
  }
};
template <>
struct Candidate<false> {
  typedef uint64_t Word;
  static __device__ __forceinline__ Word make(uint32_t key, int e) {
    return key ? ((uint64_t)key << 32) | (0xFFFFFFFFu - (uint32_t)e) : 0ull;
  }
  static __device__ __forceinline__ uint32_t key(Word w) { return (uint32_t)(w >> 32); }
  static __device__ __forceinline__ int expert(Word w) {
    return (int)(0xFFFFFFFFu - (uint32_t)w);
  }
  static __device__ __forceinline__ Word warp_max(Word w) {
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(w >> 32));
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu,
                                          (uint32_t)(w >> 32) == hi ? (uint32_t)w : 0u);
    return ((uint64_t)hi << 32) | lo;
  }
};

// v[0..N) (N a power of two) into descending order: Batcher's odd-even merge
// sort.  Stage P, step K compares i with i + K where both lie in one run of
// 2 P; templates, so that every index is known when it is compiled.
template <int N, int P, int K, typename W>
__device__ __forceinline__ void sort_step(W* v) {
#pragma unroll
  for (int i = 0; i + K < N; ++i)
    if (i >= K % P && (i - K % P) / K % 2 == 0 && i / (2 * P) == (i + K) / (2 * P)) {
      const W a = v[i], b = v[i + K];
      v[i] = a > b ? a : b;
      v[i + K] = a > b ? b : a;
    }
  if constexpr (K > 1) sort_step<N, P, K / 2>(v);
}
template <int N, int P = 1, typename W>
__device__ __forceinline__ void sort_descending(W* v) {
  if constexpr (P < N) {
    sort_step<N, P, P>(v);
    sort_descending<N, P * 2>(v);
  }
}

// One token by one warp: lane l holds experts l, l + 32, ...  Writes its
// experts and gates and enters it into the masks as token `bit` of the block.
// Each lane sorts its experts once; a round then takes the largest of the 32
// heads and the lane that had it moves up, so that a round costs EPL moves
// instead of a search through the lane's experts (16384 tokens, 256 experts,
// K = 8: 945 instructions per token before, and 26 us).
template <int EPL, bool BF16>
__device__ __forceinline__ void select_token(const RouteParams& p, int64_t t, int bit, int words,
                                             uint32_t* mask, int lane) {
  typedef Candidate<BF16> C;
  typename C::Word v[EPL];
  float x[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = j * 32 + lane;
    x[j] = e < p.E ? logit_at<BF16>(p.logits, t * p.E + e) : -INFINITY;
    if (!(x[j] > -INFINITY)) x[j] = -INFINITY;        // NaN is masked too
    v[j] = C::make(order_key(x[j]), e);
  }
  sort_descending<EPL>(v);
  typename C::Word top = C::warp_max(v[0]);
  const float m = key_value(C::key(top));
  float all = 0.0f;
  if (!p.renorm) {
    // exp by its power of two: the differences are exact where they are small,
    // so the terms that make up the sum keep their last bits
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      all += x[j] == m ? 1.0f : exp2f((x[j] - m) * 1.44269504f);
    all = farn::warp_sum(all);
  }
  typename C::Word mine = 0;
  for (int k = 0; k < p.K && top; ++k) {
    if (lane == k) mine = top;
    const bool won = v[0] == top;
#pragma unroll
    for (int j = 0; j + 1 < EPL; ++j) v[j] = won ? v[j + 1] : v[j];
    if (won) v[EPL - 1] = 0;
    top = C::warp_max(v[0]);
  }
  const float w = mine ? weight_of(C::key(mine), m) : 0.0f;
  const float total = p.renorm ? farn::warp_sum(w) : all;
  if (lane < p.K) {
    const int e = mine ? C::expert(mine) : -1;
    p.experts[t * p.K + lane] = e;
    p.gates[t * p.K + lane] = mine ? w / total : 0.0f;
    if (mine) atomicOr(&mask[e * words + (bit >> 5)], 1u << (bit & 31));
  }
}

__device__ __forceinline__ int count_bits(const uint32_t* mask, int words) {
  int c = 0;
  for (int w = 0; w < words; ++w) c += __popc(mask[w]);
  return c;
}

// Exclusive scan of v[0..n) (n <= kMaxE) in place by the whole block of
// NT threads; v[n] gets the total.  ws: 33 ints.
template <int NT>
__device__ __forceinline__ void block_scan(int32_t* v, int n, int32_t* ws) {
  constexpr int PER = (kMaxE + NT - 1) / NT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t x[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int k = tid * PER + i;
    x[i] = k < n ? v[k] : 0;
    sum += x[i];
  }
  int32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) ws[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int32_t y = lane < NT / 32 ? ws[lane] : 0, z = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xFFFFFFFFu, z, o);
      if (lane >= o) z += u;
    }
    ws[lane] = z - y;
    if (lane == 31) ws[32] = z;
  }
  __syncthreads();
  int32_t at = ws[warp] + inc - sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int k = tid * PER + i;
    if (k < n) v[k] = at;
    at += x[i];
  }
  if (tid == 0) v[n] = ws[32];
  __syncthreads();
}

// The slots of the block's pairs: base[e] is the slot of the block's first
// pair of expert e.
__device__ __forceinline__ void place(const RouteParams& p, int64_t t0, int n, int words,
                                      const uint32_t* mask, const int32_t* base) {
  for (int i = threadIdx.x; i < n * p.K; i += blockDim.x) {
    const int bit = i / p.K;
    const int64_t at = t0 * p.K + i;
    const int e = p.experts[at];
    int slot = -1;
    if (e >= 0) {
      const uint32_t* m = mask + e * words;
      int rank = __popc(m[bit >> 5] & ((1u << (bit & 31)) - 1u));
      for (int w = 0; w < (bit >> 5); ++w) rank += __popc(m[w]);
      slot = base[e] + rank;
      p.rows[slot] = (int32_t)(t0 + bit);
    }
    p.index[at] = slot;
  }
}

template <int EPL, bool BF16>
__device__ __forceinline__ void select_block(const RouteParams& p, int64_t t0, int n, int words,
                                             uint32_t* mask) {
  for (int i = threadIdx.x; i < p.E * words; i += blockDim.x) mask[i] = 0u;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n; i += kWarps)
    select_token<EPL, BF16>(p, t0 + i, i, words, mask, lane);
  __syncthreads();
}

// All tokens in one cluster: dynamic shared memory holds the masks
// [E][words], the block's counts [E] and the bases [E + 1].
template <int EPL, bool BF16>
__global__ void __launch_bounds__(kThreads) route_cluster_kernel(const RouteParams p) {
  extern __shared__ uint32_t sm[];
  __shared__ int32_t ws[33];
  farn::pdl_wait();
  farn::pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
  const int words = p.tb / 32;
  uint32_t* mask = sm;
  int32_t* count = reinterpret_cast<int32_t*>(sm + p.E * words);
  int32_t* base = count + p.E;
  const int64_t t0 = (int64_t)rank * p.tb;
  const int n = (int)max((int64_t)0, min((int64_t)p.tb, p.T - t0));
  select_block<EPL, BF16>(p, t0, n, words, mask);
  for (int e = threadIdx.x; e < p.E; e += kThreads) count[e] = count_bits(mask + e * words, words);
  cluster.sync();
  int before[(kMaxE + kThreads - 1) / kThreads];
#pragma unroll
  for (int i = 0; i < (kMaxE + kThreads - 1) / kThreads; ++i) {
    const int e = threadIdx.x + i * kThreads;
    if (e >= p.E) break;
    int total = 0;
    before[i] = 0;
    for (int r = 0; r < size; ++r) {
      if (r == rank) before[i] = total;
      total += cluster.map_shared_rank(count, r)[e];
    }
    base[e] = total;
  }
  cluster.sync();     // the counts are read: no block leaves before that
  block_scan<kThreads>(base, p.E, ws);
  if (rank == 0)
    for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = base[e];
  const int64_t live = base[p.E];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < (kMaxE + kThreads - 1) / kThreads; ++i) {
    const int e = threadIdx.x + i * kThreads;
    if (e < p.E) base[e] += before[i];
  }
  __syncthreads();
  place(p, t0, n, words, mask, base);
  // slots of pairs that chose no expert
  for (int64_t s = live + (int64_t)rank * kThreads + threadIdx.x; s < p.T * p.K;
       s += (int64_t)size * kThreads)
    p.rows[s] = -1;
}

// Where a block's counts lie between the kernels of a long call: no memory
// is needed beyond the outputs.  A block's own part of `index` holds them (and
// later its bases) until the block writes the index there; the last block,
// whose part may be shorter than E, uses the start of `rows`, and takes its
// bases from the offsets.  The host sees to tb * K >= E and nb >= 2.
__device__ __forceinline__ int32_t* counts_of(const RouteParams& p, int b) {
  return b + 1 < p.nb ? p.index + (int64_t)b * p.tb * p.K : p.rows;
}
__device__ __forceinline__ int tokens_of(const RouteParams& p, int b) {
  return b + 1 < p.nb ? p.tb : (int)(p.T - (int64_t)b * p.tb);
}

template <int EPL, bool BF16>
__global__ void __launch_bounds__(kThreads) route_select_kernel(const RouteParams p) {
  extern __shared__ uint32_t sm[];
  farn::pdl_wait();
  farn::pdl_trigger();
  const int b = blockIdx.x, n = tokens_of(p, b), words = (n + 31) / 32;
  select_block<EPL, BF16>(p, (int64_t)b * p.tb, n, words, sm);
  int32_t* count = counts_of(p, b);
  for (int e = threadIdx.x; e < p.E; e += kThreads) count[e] = count_bits(sm + e * words, words);
}

// One cluster: each CTA scans the blocks' counts of its share of the
// experts, the totals meet in distributed shared memory.
__global__ void __launch_bounds__(kScanThreads) __cluster_dims__(kScanCtas, 1, 1)
route_scan_kernel(const RouteParams p) {
  constexpr int kGroups = kScanThreads / 32;        // runs of blocks, one per warp
  __shared__ int32_t part[kGroups][kScanE];
  __shared__ int32_t total[kMaxE + 1];
  __shared__ int32_t ws[33];
  farn::cluster_arrive_release();     // this CTA runs: the others may write to its memory
  farn::pdl_wait();
  farn::pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // 32 experts, a lane each, to a CTA if there are CTAs enough
  const int share = max(32, (p.E + kScanCtas - 1) / kScanCtas), e0 = rank * share;
  const int e1 = min(p.E, e0 + share), per = (p.nb + kGroups - 1) / kGroups;
  const int b0 = warp * per, b1 = min(p.nb, b0 + per);
  for (int i = lane; e0 + i < e1; i += 32) {
    int32_t sum = 0;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) sum += counts_of(p, b)[e0 + i];
    part[warp][i] = sum;
  }
  __syncthreads();
  farn::cluster_wait_acquire();       // all CTAs run
  if (e0 + (int)threadIdx.x < e1) {
    int32_t sum = 0;
    for (int w = 0; w < kGroups; ++w) {
      const int32_t x = part[w][threadIdx.x];
      part[w][threadIdx.x] = sum;
      sum += x;
    }
    for (int r = 0; r < kScanCtas; ++r)
      cluster.map_shared_rank(total, r)[e0 + threadIdx.x] = sum;
  }
  cluster.sync();
  block_scan<kScanThreads>(total, p.E, ws);
  if (rank == 0)
    for (int e = threadIdx.x; e <= p.E; e += kScanThreads) p.offsets[e] = total[e];
  for (int i = lane; e0 + i < e1; i += 32) {
    int32_t at = total[e0 + i] + part[warp][i];
#pragma unroll 8
    for (int b = b0; b < min(b1, p.nb - 1); ++b) {
      int32_t* c = counts_of(p, b) + e0 + i;
      const int32_t x = *c;
      *c = at;
      at += x;
    }
  }
}

__global__ void __launch_bounds__(kThreads) route_place_kernel(const RouteParams p) {
  extern __shared__ uint32_t sm[];
  farn::pdl_wait();
  farn::pdl_trigger();
  const int b = blockIdx.x, n = tokens_of(p, b), words = (n + 31) / 32;
  const int64_t t0 = (int64_t)b * p.tb;
  uint32_t* mask = sm;
  int32_t* base = reinterpret_cast<int32_t*>(sm + p.E * words);
  for (int i = threadIdx.x; i < p.E * words; i += kThreads) mask[i] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < n * p.K; i += kThreads) {
    const int bit = i / p.K, e = p.experts[t0 * p.K + i];
    if (e >= 0) atomicOr(&mask[e * words + (bit >> 5)], 1u << (bit & 31));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads)
    base[e] = b + 1 < p.nb ? counts_of(p, b)[e]
                           : p.offsets[e + 1] - count_bits(mask + e * words, words);
  __syncthreads();
  place(p, t0, n, words, mask, base);
  const int64_t live = p.offsets[p.E];
  for (int64_t s = live + (int64_t)b * kThreads + threadIdx.x; s < p.T * p.K;
       s += (int64_t)p.nb * kThreads)
    p.rows[s] = -1;
}

typedef void (*RouteKernel)(const RouteParams);

template <int EPL>
RouteKernel pick_epl(bool cluster, bool bf16) {
  if (cluster) return bf16 ? &route_cluster_kernel<EPL, true> : &route_cluster_kernel<EPL, false>;
  return bf16 ? &route_select_kernel<EPL, true> : &route_select_kernel<EPL, false>;
}

// EPL: experts per lane of the selecting warp
RouteKernel pick(int E, bool cluster, bool bf16) {
  if (E <= 64) return pick_epl<2>(cluster, bf16);
  if (E <= 128) return pick_epl<4>(cluster, bf16);
  if (E <= 256) return pick_epl<8>(cluster, bf16);
  if (E <= 512) return pick_epl<16>(cluster, bf16);
  return pick_epl<32>(cluster, bf16);
}

constexpr int kClusterTokens = 64;    // tokens per block of the one-cluster kernel
constexpr int kClusterMax = 8;        // its largest cluster
constexpr int64_t kMaxTokens = 1024;  // most tokens per block of the long calls

size_t cluster_smem(int E, int tb) { return (size_t)(E * (tb / 32) + 2 * E + 1) * 4; }
size_t block_smem(int E, int tokens) { return (size_t)(E * ((tokens + 31) / 32) + E) * 4; }

int run(RouteKernel k, unsigned grid, unsigned cluster, size_t smem, const farn_ctx* ctx,
        const RouteParams& p, unsigned threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  unsigned n = 0;
  if (cluster) {
    attrs[n].id = cudaLaunchAttributeClusterDimension;
    attrs[n].val.clusterDim.x = cluster;
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
  if (cudaLaunchKernelEx(&cfg, k, p) != cudaSuccess) {
    cudaGetLastError();
    return FARN_ERR_CUDA;
  }
  return FARN_OK;
}

}  // namespace

namespace farn_host {

// Shared-memory opt-in of the router's kernels, on the current device.
bool route_setup(const farn_ctx* ctx) {
  for (int E : {64, 128, 256, 512, 1024})
    for (int i = 0; i < 4; ++i) {
      const void* k = (const void*)pick(E, i & 1, i & 2);
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, k) != cudaSuccess ||
          cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               ctx->max_smem - (int)fa.sharedSizeBytes) != cudaSuccess)
        return false;
    }
  cudaFuncAttributes fa;
  return cudaFuncSetAttribute((const void*)route_place_kernel,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, ctx->max_smem) ==
             cudaSuccess &&
         cudaFuncGetAttributes(&fa, (const void*)route_scan_kernel) == cudaSuccess;
}

}  // namespace farn_host

extern "C" int farn_moe_route(const farn_ctx* ctx, const void* logits, int logits_dtype,
                              int64_t T, int E, int K, int renormalize, int32_t* experts,
                              float* gates, int32_t* index, int32_t* rows, int32_t* offsets,
                              cudaStream_t stream) {
  if (!ctx || (logits_dtype != FARN_BF16 && logits_dtype != FARN_F32) || T < 0 || E < 1 ||
      E > FARN_MAX_EXPERTS || K < 1 || K > FARN_MAX_W || K > E)
    return FARN_ERR_INVALID_ARG;
  if (T > 0x7FFFFFFF / K) return FARN_ERR_INVALID_ARG;   // slots are 32-bit numbers
  if (!offsets || ((uintptr_t)offsets & 3u)) return FARN_ERR_INVALID_ARG;
  const int64_t lb = T * E * (logits_dtype == FARN_BF16 ? 2 : 4), pb = T * K * 4;
  const void* outs[5] = {experts, gates, index, rows, offsets};
  const int64_t bytes[5] = {pb, pb, pb, pb, (int64_t)(E + 1) * 4};
  if (T > 0) {
    if (!logits || ((uintptr_t)logits & (logits_dtype == FARN_BF16 ? 1u : 3u)))
      return FARN_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)
      if (!outs[i] || ((uintptr_t)outs[i] & 3u)) return FARN_ERR_INVALID_ARG;
    for (int i = 0; i < 5; ++i) {
      if (overlaps(outs[i], bytes[i], logits, lb)) return FARN_ERR_ALIAS;
      for (int j = i + 1; j < 5; ++j)
        if (overlaps(outs[i], bytes[i], outs[j], bytes[j])) return FARN_ERR_ALIAS;
    }
  }
  if (ctx->fault_launch || !ctx->route_ok) return FARN_ERR_CUDA;

  RouteParams p;
  p.logits = logits;
  p.T = T;
  p.E = E;
  p.K = K;
  p.renorm = renormalize != 0;
  p.experts = experts;
  p.gates = gates;
  p.index = index;
  p.rows = rows;
  p.offsets = offsets;
  const bool bf16 = logits_dtype == FARN_BF16;
  DeviceGuard dg(ctx->device);
  if (!dg.ok) { cudaGetLastError(); return FARN_ERR_CUDA; }

  // Long calls: a block's part of `index` has to hold E counts, and a few
  // hundred blocks keep the scan short.
  int64_t tb = 64;
  while (tb < kMaxTokens && (tb * K < E || T / tb > 512)) tb *= 2;
  if (T <= kClusterTokens * kClusterMax || T <= tb) {
    unsigned c = 1;
    while (c < (unsigned)kClusterMax && (int64_t)c * 16 < T) c *= 2;
    p.tb = (int)((T + c - 1) / c + 31) / 32 * 32;
    if (p.tb < 32) p.tb = 32;
    p.nb = (int)c;
    return run(pick(E, true, bf16), c, c, cluster_smem(E, p.tb), ctx, p, kThreads, stream);
  }
  p.tb = (int)tb;
  p.nb = (int)((T + tb - 1) / tb);
  const size_t smem = block_smem(E, p.tb);
  int st = run(pick(E, false, bf16), (unsigned)p.nb, 0, smem, ctx, p, kThreads, stream);
  if (st == FARN_OK)
    st = run(&route_scan_kernel, kScanCtas, 0, 0, ctx, p, kScanThreads, stream);
  if (st == FARN_OK)
    st = run(&route_place_kernel, (unsigned)p.nb, 0, smem, ctx, p, kThreads, stream);
  return st;
}

// Query and key heads: RMSNorm of every head and its rotation by position in
// one pass over the projection's output, keys and values going to bf16 or
// straight into a paged cache in 8 or 4 bits; and the cache read back.
//
//   y = x / sqrt(mean(x^2) + eps) * w         (x as it is without a weight)
//   (a, b) -> (a cos - b sin, b cos + a sin)  for R / 2 pairs of a head's first
//                                             R elements, by the angle
//                                             positions[axis of the pair] * freq
//
// in fp32, one rounding at the end.  A row is a token's head: 8 elements per
// lane on 8, 16 or 32 lanes (D <= 64, 128, 256), so the sum of squares and a row's
// amax are shuffles within the row's lanes.  A warp keeps one token's angles in
// registers for all the heads it takes.
// Memory bound for long calls, one launch and two dependent loads for short
// ones.
//
// The angle: the frequency in turns as a 64-bit fixed-point fraction, times
// the position modulo 2^64, is the angle's place in the turn to 2^-32 however
// far the position is (fp32 angles lose 6e-8 of the position, 0.06 radians at
// 10^6; fp64 runs at 1/64 rate).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "farn.h"
#include "farn_fp8.cuh"
#include "farn_internal.h"

using farn_host::DeviceGuard;
using farn_host::aligned16;
using farn_host::overlaps;
using farn_host::product_fits;

namespace {

constexpr int kThreads = 128;         // of the kernel for any head size
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;             // rows per lane group whose loads are in flight
// CTAs per SM, of a warp each: warps have nothing in common, and one that is done
// makes room at once (four to a CTA: 8192 tokens of 40 and 8 heads of 128 47.5 us, now
// 46.9; 4099 of 16 and 16 of 80 15.8, now 15.3; 2048 of 8 written 6.2, now 5.5).  28
// leave a thread 72 registers, and all instances but one spill (16 to 172 bytes of
// loads); 25 to 32 CTAs with 2 to 6 rows ahead were no faster.
constexpr int kCtas = 28;
constexpr int kMaxDim = 1024;
constexpr int kMaxAxes = 4;

struct Cache {
  uint8_t *codes[2];                  // keys, values
  void *scale[2];                     // fp32 per row, or E4M3 per 16 elements
  float g[2];                         // NVFP4: tensor scales
  int64_t slots;
};

struct HeadsParams {
  const uint16_t *in[3];              // queries, keys, values
  int64_t in_stride[3];               // elements from one token to the next
  uint16_t *out[2];                   // queries, keys (unless they go to the cache)
  int64_t out_stride[2];
  const uint16_t *weight[2];
  int heads[3];
  int D, R;
  bool interleaved;
  float eps;
  const int32_t *positions;           // [axes, T]
  const float *freqs;                 // [R / 2]
  int axis_end[kMaxAxes];             // first pair after each axis's
  int64_t T;
  Cache cache;
  const int32_t *slots;               // [T]
  int groups;                         // tasks that share a token's rows
};

// positions' turn fraction: freq / (2 pi) * 2^64 modulo 2^64, to its last bit
// but one for frequencies up to 2^8.
__device__ __forceinline__ uint64_t turn_step(float freq) {
  constexpr uint64_t kC = 0xA2F9836E4E44152Aull;      // 2^66 / (2 pi)
  const uint32_t b = __float_as_uint(freq);
  const int ex = (int)((b >> 23) & 255u) - 150;       // freq = m * 2^ex
  const uint64_t m = (b & 0x7FFFFFu) | 0x800000u;
  if ((b & 0x7F800000u) == 0u) return 0ull;           // below 2^-126
  const uint64_t hi = __umul64hi(m, kC), lo = m * kC;
  const int sh = ex - 2;
  uint64_t f;
  if (sh >= 64) f = 0ull;
  else if (sh >= 0) f = lo << sh;
  else if (sh > -64) f = (hi << (64 + sh)) | (lo >> -sh);
  else f = sh > -128 ? hi >> (-sh - 64) : 0ull;
  return (b >> 31) ? 0ull - f : f;
}
__device__ __forceinline__ void sincos_at(int32_t pos, uint64_t step, float* s, float* c) {
  // The place in the turn: the nearest quarter, and what is left in fp32, at most
  // an eighth of a turn (a whole turn's place in 24 bits would be off four times
  // as far).
  const uint32_t top = (uint32_t)(((uint64_t)(int64_t)pos * step) >> 32);
  const uint32_t quarter = (top + 0x20000000u) >> 30;
  const int32_t left = (int32_t)(top - (quarter << 30));
  float a, b;
  sincospif((float)left * 4.656612873077393e-10f, &a, &b);       // 2^-31 half turns
  const float u = quarter & 1u ? b : a, v = quarter & 1u ? a : b;
  *s = quarter & 2u ? -u : u;
  *c = (quarter + 1u) & 2u ? -v : v;
}
__device__ __forceinline__ int axis_of(const HeadsParams& p, int pair) {
  int a = 0;
#pragma unroll
  for (int i = 0; i < kMaxAxes - 1; ++i) a += pair >= p.axis_end[i];
  return a;
}

// Where a lane's 8 elements of a row lie: two runs of four, elements [a, a + 4) and
// [b, b + 4).
//
// Contiguous (b = a + 4): unrotated rows, and pairs of neighbours.  Halved: a lane
// of the first R / 8 has the first and the second elements of four pairs, so that
// a pair never leaves its lane and its angle is computed once; the others have
// what follows the rotated part.  (With 8 neighbouring elements per lane a pair's
// partner was 8 shuffles away: 8192 tokens of 40 and 8 heads of 128 took 96 us.)
struct Runs {
  int a, b;
};
__device__ __forceinline__ Runs contiguous(int l) { return Runs{l * 8, l * 8 + 4}; }
__device__ __forceinline__ Runs halved(int l, int R) {
  return l < R / 8 ? Runs{l * 4, R / 2 + l * 4} : contiguous(l);
}

// A row of the cache from a lane's 8 values; every lane of the warp calls it.
// row: slot * heads + head.  live: the row and the lane's elements exist.  half:
// the lane's runs lie in two halves of the row (NVFP4: all of the row's lanes' do,
// and a block of 16 elements is a run of four lanes).
template <int FMT, int L>
__device__ __forceinline__ void store_cache8(const Cache& c, int which, int64_t row, int D,
                                             const Runs& r, int l, bool half, const float* x,
                                             bool live) {
  if constexpr (FMT == FARN_CACHE_FP8) {
    float m = farn::amax8(x);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const farn::Fp8Scale s = farn::fp8_scale(m);
    if (!live) return;
    const uint2 w = farn::fp8_codes8(x, s.inv);
    uint8_t* to = c.codes[which] + row * D;
    *reinterpret_cast<uint32_t*>(to + r.a) = w.x;
    *reinterpret_cast<uint32_t*>(to + r.b) = w.y;
    if (l == 0) static_cast<float*>(c.scale[which])[row] = s.scale;
  } else {
    // as nvfp4_vec, from fp32 values
    float m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) m[i] = fmaxf(m[i], fabsf(x[4 * i + e]));
    }
    if (half) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
    } else {
      m[0] = fmaxf(m[0], m[1]);
      m[0] = m[1] = fmaxf(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
    }
    uint8_t* to = c.codes[which] + row * (D / 2);
    uint8_t* scale = static_cast<uint8_t*>(c.scale[which]) + row * (D / 16);
    const float g = c.g[which];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t s = farn::pack_e4m3x2((m[i] / 6.0f) * g, 0.0f) & 0xFFu;
      const float sv = farn::e4m3_to_f32(s), inv = g / sv;
      uint32_t w = 0u;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w |= farn::pack_e2m1x2(fminf(x[4 * i + 2 * e] * inv, 6.0f),
                               fminf(x[4 * i + 2 * e + 1] * inv, 6.0f))
             << (8 * e);
      if (!live) continue;
      const int at = i ? r.b : r.a;
      *reinterpret_cast<uint16_t*>(to + at / 2) = (uint16_t)(sv > 0.0f ? w : 0u);
      if (half ? (l & 3) == 0 : (l & 1) == 0 && i == 0) scale[at / 16] = (uint8_t)s;
    }
  }
}

// What a lane keeps for all the rows of one role (0 queries, 1 keys, 2 values)
// that its warp takes.
struct Turn {
  float c[4], s[4];
  int pairs;                          // how many of its four turn
};

// The passes [lo, hi) of a role and token: kRows rows each, one per L lanes.
// FMT: the cache's format, or 0: keys go to out[1].  HALF: pairs lie in halves.
// The code is about instructions: with roles, layouts and addresses worked out
// per row 8192 tokens of 40 and 8 heads of 128 took 77 us, 260 instructions to a
// pass, two thirds of the issue slots; it takes 47 with 170.  What bounds it now is
// latency: of the 9.3 cycles that a warp takes per instruction 3.1 wait for memory,
// and 25 warps per SM leave a third of the issue slots empty.  (One loop for all roles: 50;
// the rows brought ahead of the warps through shared memory: 62; a token's angles
// shared by four warps: 55; four rows' sums joined together: 53, for the registers.)
template <int ROLE, int L, int FMT, bool HALF>
__device__ __forceinline__ void run_role(const HeadsParams& p, int64_t t, int lo, int hi, int l,
                                         int sub, const uint2* weight, const Turn& turn,
                                         int64_t slot, float inv_d) {
  constexpr int kRows = 32 / L;
  constexpr bool kTurned = ROLE < 2, kCached = FMT != 0 && ROLE > 0;
  if (lo >= hi || (kCached && slot < 0)) return;
  const int heads = p.heads[ROLE], D = p.D;
  const Runs r = HALF && kTurned ? halved(l, p.R) : contiguous(l);
  const int head0 = lo * kRows + sub;
  // lanes without elements read and write nothing
  const int end = l * 8 < D ? min(heads, hi * kRows) : 0;
  const int step = kRows * D;
  const uint16_t* in = p.in[ROLE] + t * p.in_stride[ROLE] + (int64_t)head0 * D;
  uint16_t* out = nullptr;
  if (!kCached) out = p.out[ROLE < 2 ? ROLE : 0] + t * p.out_stride[ROLE < 2 ? ROLE : 0] +
                      (int64_t)head0 * D;
  const bool norm = kTurned && p.weight[ROLE < 2 ? ROLE : 0] != nullptr;
  float w[8];
  if (kTurned) farn::unpack8(make_uint4(weight[0].x, weight[0].y, weight[1].x, weight[1].y), w);
  for (int n = lo, head = head0; n < hi; n += kAhead) {
    uint2 raw[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
      if (head + i * kRows < end) {
        raw[i][0] = *reinterpret_cast<const uint2*>(in + i * step + r.a);
        raw[i][1] = *reinterpret_cast<const uint2*>(in + i * step + r.b);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (n + i >= hi) break;
      float x[8];
      farn::unpack8(make_uint4(raw[i][0].x, raw[i][0].y, raw[i][1].x, raw[i][1].y), x);
      if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float rstd = __frsqrt_rn(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (x[e] * rstd) * w[e];
      }
      if (kTurned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float& a = x[HALF ? e : 2 * e];
          float& b = x[HALF ? e + 4 : 2 * e + 1];
          if (e < turn.pairs) {
            const float ya = a * turn.c[e] - b * turn.s[e];
            b = b * turn.c[e] + a * turn.s[e];
            a = ya;
          }
        }
      }
      const int h = head + i * kRows;
      if constexpr (!kCached) {
        if (h < end) {
          const uint4 v = farn::pack8(x);
          *reinterpret_cast<uint2*>(out + i * step + r.a) = make_uint2(v.x, v.y);
          *reinterpret_cast<uint2*>(out + i * step + r.b) = make_uint2(v.z, v.w);
        }
      } else {
        store_cache8<FMT, L>(p.cache, ROLE - 1, slot * heads + h, D, r, l, HALF && kTurned, x,
                             h < end);
      }
    }
    head += kAhead * kRows;
    in += kAhead * step;
    if (!kCached) out += kAhead * step;
  }
}

template <int L, int FMT, bool HALF>
__global__ void __launch_bounds__(32, kCtas)
heads_kernel(const __grid_constant__ HeadsParams p) {
  constexpr int kRows = 32 / L;                       // rows of a pass
  farn::pdl_wait();
  farn::pdl_trigger();
  const int l = threadIdx.x % L, sub = threadIdx.x / L;
  const int passes_q = (p.heads[0] + kRows - 1) / kRows;
  const int passes_k = (p.heads[1] + kRows - 1) / kRows;
  const int passes_v = (p.heads[2] + kRows - 1) / kRows;
  const int turned = passes_q + passes_k, passes = turned + passes_v;
  const int per = (passes + p.groups - 1) / p.groups;
  // this lane's pairs: the four from 4 l on, or fewer
  const int pair0 = l * 4;
  Turn turn;
  turn.pairs = min(max(p.R / 2 - pair0, 0), 4);
  const Runs r = HALF ? halved(l, p.R) : contiguous(l);
  uint64_t step[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) step[i] = i < turn.pairs ? turn_step(p.freqs[pair0 + i]) : 0ull;
  uint2 weight[2][2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const bool have = l * 8 < p.D && p.heads[w] && p.weight[w];
    weight[w][0] = have ? __ldg(reinterpret_cast<const uint2*>(p.weight[w] + r.a))
                        : make_uint2(0u, 0u);
    weight[w][1] = have ? __ldg(reinterpret_cast<const uint2*>(p.weight[w] + r.b))
                        : make_uint2(0u, 0u);
  }
  const float inv_d = 1.0f / (float)p.D;
  const int64_t tasks = p.T * p.groups;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int64_t t = p.groups == 1 ? task : task / p.groups;
    const int first = (int)(task - t * p.groups) * per, end = min(first + per, passes);
    int64_t slot = 0;
    if (FMT != 0) {
      slot = p.slots[t];
      if (slot >= p.cache.slots) slot = -1;
    }
    if (first < turned && p.R > 0) {
      const int a0 = axis_of(p, pair0);
      const int32_t at0 = turn.pairs > 0 ? p.positions[a0 * p.T + t] : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        turn.c[i] = 1.0f;
        turn.s[i] = 0.0f;
        if (i < turn.pairs) {
          const int a = axis_of(p, pair0 + i);
          sincos_at(a == a0 ? at0 : p.positions[a * p.T + t], step[i], &turn.s[i], &turn.c[i]);
        }
      }
    }
    run_role<0, L, FMT, HALF>(p, t, first, min(end, passes_q), l, sub, weight[0], turn, slot,
                              inv_d);
    run_role<1, L, FMT, HALF>(p, t, max(first - passes_q, 0), min(end, turned) - passes_q, l, sub,
                              weight[1], turn, slot, inv_d);
    if (FMT != 0)
      run_role<2, L, FMT, HALF>(p, t, max(first - turned, 0), end - turned, l, sub, nullptr, turn,
                                slot, inv_d);
  }
}

// Any head size up to kMaxDim, any alignment: a warp per row, the row in
// shared memory.
template <int FMT>
__global__ void __launch_bounds__(kThreads)
heads_plain_kernel(const __grid_constant__ HeadsParams p) {
  __shared__ float rows[kWarps][kMaxDim];
  farn::pdl_wait();
  farn::pdl_trigger();
  const int lane = threadIdx.x & 31;
  float* x = rows[threadIdx.x >> 5];
  const int all = p.heads[0] + p.heads[1] + p.heads[2], D = p.D, half = p.R >> 1;
  const int64_t tasks = p.T * all;
  for (int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); task < tasks;
       task += (int64_t)gridDim.x * kWarps) {
    const int64_t t = task / all;
    int head = (int)(task - t * all), role = 0;
    while (role < 2 && head >= p.heads[role]) head -= p.heads[role++];
    int64_t slot = 0;
    if (FMT != 0 && role > 0) {
      slot = p.slots[t];
      if (slot < 0 || slot >= p.cache.slots) continue;
    }
    const uint16_t* in = p.in[role] + t * p.in_stride[role] + (int64_t)head * D;
    float ss = 0.0f;
    for (int i = lane; i < D; i += 32) {
      x[i] = farn::bf_lo(in[i]);
      ss = fmaf(x[i], x[i], ss);
    }
    if (role < 2) {
      if (p.weight[role]) {
        ss = farn::warp_sum(ss);
        const float rstd = 1.0f / sqrtf(ss / (float)D + p.eps);
        for (int i = lane; i < D; i += 32) x[i] = (x[i] * rstd) * farn::bf_lo(p.weight[role][i]);
      }
      __syncwarp();
      for (int i = lane; i < half; i += 32) {
        float s, c;
        sincos_at(p.positions[axis_of(p, i) * p.T + t], turn_step(p.freqs[i]), &s, &c);
        const int ia = p.interleaved ? 2 * i : i, ib = p.interleaved ? 2 * i + 1 : i + half;
        const float a = x[ia], b = x[ib];
        x[ia] = a * c - b * s;
        x[ib] = b * c + a * s;
      }
    }
    __syncwarp();
    if (role == 0 || (FMT == 0 && role == 1)) {
      uint16_t* out = p.out[role] + t * p.out_stride[role] + (int64_t)head * D;
      for (int i = lane; i < D; i += 32) out[i] = farn::to_bf16(x[i]);
    } else if constexpr (FMT != 0) {
      const int which = role - 1;
      const int64_t row = slot * p.heads[1] + head;
      if constexpr (FMT == FARN_CACHE_FP8) {
        float m = 0.0f;
        for (int i = lane; i < D; i += 32) m = fmaxf(m, fabsf(x[i]));
        const farn::Fp8Scale s = farn::fp8_scale(farn::warp_max(m));
        for (int i = lane; i < D; i += 32)
          p.cache.codes[which][row * D + i] = (uint8_t)farn::pack_e4m3x2(x[i] * s.inv, 0.0f);
        if (lane == 0) static_cast<float*>(p.cache.scale[which])[row] = s.scale;
      } else {
        for (int b = lane; b < D / 16; b += 32) {
          const float g = p.cache.g[which];
          float m = 0.0f;
          for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[16 * b + e]));
          const uint32_t s = farn::pack_e4m3x2((m / 6.0f) * g, 0.0f) & 0xFFu;
          const float sv = farn::e4m3_to_f32(s), inv = g / sv;
          for (int e = 0; e < 8; ++e) {
            const uint32_t w = farn::pack_e2m1x2(fminf(x[16 * b + 2 * e] * inv, 6.0f),
                                                 fminf(x[16 * b + 2 * e + 1] * inv, 6.0f));
            p.cache.codes[which][row * (D / 2) + 8 * b + e] = (uint8_t)(sv > 0.0f ? w : 0u);
          }
          static_cast<uint8_t*>(p.cache.scale[which])[row * (D / 16) + b] = (uint8_t)s;
        }
      }
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------- reading back
struct ReadParams {
  Cache cache;
  int heads, D, page_size;
  int64_t pages;
  const int32_t *table;               // [B, width]
  int B;
  int64_t width;
  const int32_t *offsets;             // [B + 1]
  int64_t tokens;
  uint16_t *out[2];
};

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 4;        // per warp, or part of a warp that has a token
constexpr int kReadAhead = 4;         // vectors per lane, of keys and of values, in flight
constexpr int kPlainTokens = 8;       // per CTA of the scalar kernel

// The cache slot of output token n: -1 where its page does not exist, -2
// where no sequence has it.
__device__ __forceinline__ int64_t slot_of(const ReadParams& p, int64_t n) {
  if (n >= p.tokens || n < p.offsets[0] || n >= p.offsets[p.B]) return -2;
  int lo = 0, hi = p.B - 1;           // the last sequence that starts at n or before
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.offsets[mid] <= n) lo = mid; else hi = mid - 1;
  }
  const int64_t pos = n - p.offsets[lo];
  if (pos < 0) return -2;
  const int64_t page = pos / p.page_size;
  if (page >= p.width) return -1;
  const int64_t at = p.table[lo * p.width + page];
  if (at < 0 || at >= p.pages) return -1;
  return at * p.page_size + pos % p.page_size;
}

// Eight values of a token's row of heads * D elements, from element e on.
// VEC: D a multiple of 8, codes 8-byte (NVFP4: 4-byte) aligned.
template <int FMT>
struct Piece {
  uint2 codes;
  float scale;
};
template <int FMT>
__device__ __forceinline__ Piece<FMT> load_piece(const ReadParams& p, int which, int64_t slot,
                                                 int e, int head) {
  Piece<FMT> r;
  const int64_t row = (int64_t)p.heads * p.D;
  if constexpr (FMT == FARN_CACHE_FP8) {
    r.codes = __ldg(reinterpret_cast<const uint2*>(p.cache.codes[which] + slot * row + e));
    r.scale = __ldg(static_cast<const float*>(p.cache.scale[which]) + slot * p.heads +
                    head);
  } else {
    r.codes.x =
        __ldg(reinterpret_cast<const uint32_t*>(p.cache.codes[which] + (slot * row + e) / 2));
    r.codes.y = 0u;
    r.scale = __uint_as_float(
        (uint32_t)__ldg(static_cast<const uint8_t*>(p.cache.scale[which]) + (slot * row + e) / 16));
  }
  return r;
}
template <int FMT>
__device__ __forceinline__ uint4 piece_values(const ReadParams& p, int which, const Piece<FMT>& r) {
  float x[8];
  if constexpr (FMT == FARN_CACHE_FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t two = (i < 2 ? r.codes.x : r.codes.y) >> (16 * (i & 1)) & 0xFFFFu;
      const float2 f = farn::e4m3x2_to_f32(two);
      x[2 * i] = f.x * r.scale;
      x[2 * i + 1] = f.y * r.scale;
    }
  } else {
    const float s = farn::e4m3_to_f32(__float_as_uint(r.scale)) / p.cache.g[which];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = farn::e2m1x2_to_f32((r.codes.x >> (8 * i)) & 0xFFu);
      x[2 * i] = f.x * s;
      x[2 * i + 1] = f.y * s;
    }
  }
  return farn::pack8(x);
}

// LPT lanes to a token, 8 elements each at a time: a lane's places in the row, and
// with them its heads, are the same for all its tokens.  Memory bound: 115810
// tokens of 8 heads of 128 in 8 bits take 110 us, 6.5 TB/s (147 with a block per 8
// tokens and places worked out for every vector).
template <int FMT, int LPT>
__global__ void __launch_bounds__(kReadThreads)
cache_read_kernel(const __grid_constant__ ReadParams p) {
  farn::pdl_wait();
  farn::pdl_trigger();
  constexpr int kSubs = 32 / LPT;
  const int lane = threadIdx.x & 31, l = lane % LPT, sub = lane / LPT;
  const int row = p.heads * p.D, vecs = row / 8;
  const int64_t n0 =
      ((int64_t)blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5)) * (kSubs * kReadTokens);
  if (n0 >= p.tokens) return;
  // lane i looks up token n0 + i
  const int64_t mine = lane < kSubs * kReadTokens ? slot_of(p, n0 + lane) : -2;
  for (int v0 = 0; v0 < vecs; v0 += LPT * kReadAhead) {
    int head[kReadAhead];
#pragma unroll
    for (int j = 0; j < kReadAhead; ++j) head[j] = (v0 + j * LPT + l) * 8 / p.D;
#pragma unroll 1
    for (int i = 0; i < kReadTokens; ++i) {
      const int at = i * kSubs + sub;
      const int64_t slot = __shfl_sync(0xFFFFFFFFu, mine, at);
      Piece<FMT> r[2][kReadAhead];
#pragma unroll
      for (int j = 0; j < kReadAhead; ++j) {
        const int v = v0 + j * LPT + l;
        if (v < vecs && slot >= 0) {
          r[0][j] = load_piece<FMT>(p, 0, slot, v * 8, head[j]);
          r[1][j] = load_piece<FMT>(p, 1, slot, v * 8, head[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < kReadAhead; ++j) {
        const int v = v0 + j * LPT + l;
        if (v < vecs && slot != -2) {
#pragma unroll
          for (int which = 0; which < 2; ++which) {
            uint4 o = make_uint4(0u, 0u, 0u, 0u);
            if (slot >= 0) o = piece_values<FMT>(p, which, r[which][j]);
            *reinterpret_cast<uint4*>(p.out[which] + (n0 + at) * row + v * 8) = o;
          }
        }
      }
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kReadThreads)
cache_read_plain_kernel(const __grid_constant__ ReadParams p) {
  __shared__ int64_t slots[kPlainTokens];
  farn::pdl_wait();
  farn::pdl_trigger();
  const int64_t n0 = (int64_t)blockIdx.x * kPlainTokens;
  if (threadIdx.x < kPlainTokens) slots[threadIdx.x] = slot_of(p, n0 + threadIdx.x);
  __syncthreads();
  const int row = p.heads * p.D, total = kPlainTokens * 2 * row;
  for (int i = threadIdx.x; i < total; i += kReadThreads) {
    const int t = i / (2 * row), v = i - t * 2 * row, which = v >= row, e = v - which * row;
    const int64_t slot = slots[t];
    if (slot == -2) continue;
    float x = 0.0f;
    if (slot >= 0) {
      const int64_t at = slot * row + e;
      if constexpr (FMT == FARN_CACHE_FP8) {
        x = farn::e4m3_to_f32(p.cache.codes[which][at]) *
            static_cast<const float*>(p.cache.scale[which])[slot * p.heads + e / p.D];
      } else {
        const float2 f = farn::e2m1x2_to_f32(p.cache.codes[which][at / 2]);
        x = ((at & 1) ? f.y : f.x) *
            (farn::e4m3_to_f32(static_cast<const uint8_t*>(p.cache.scale[which])[at / 16]) /
             p.cache.g[which]);
      }
    }
    p.out[which][(n0 + t) * row + e] = farn::to_bf16(x);
  }
}

// -------------------------------------------------------------------- host
template <typename K, typename P>
int launch(const farn_ctx* ctx, K kernel, int64_t grid, int threads, cudaStream_t stream,
           const P& params) {
  DeviceGuard dg(ctx->device);
  if (!dg.ok) { cudaGetLastError(); return FARN_ERR_CUDA; }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = ctx->pdl ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, params) != cudaSuccess) {
    cudaGetLastError();
    return FARN_ERR_CUDA;
  }
  return FARN_OK;
}

// T rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void* at;
  int64_t stride, width, T;
  int64_t span() const { return at && T > 0 ? (T - 1) * stride + width : 0; }
};

// Rows of one stride may lie between each other's (heads of one projection's
// output); rows of different strides overlap where their spans do.
bool rows_overlap(const Rows& a, const Rows& b) {
  if (!overlaps(a.at, a.span(), b.at, b.span())) return false;
  if (a.stride != b.stride || a.T < 2 || b.T < 2) return true;
  const int64_t s = a.stride;
  int64_t d = (int64_t)((intptr_t)b.at - (intptr_t)a.at) % s;
  if (d < 0) d += s;
  return d < a.width || d + b.width > s;
}

bool same_rows(const Rows& a, const Rows& b) { return a.at == b.at && a.stride == b.stride; }

bool heads_size_ok(int64_t T, int heads, int D, int64_t stride) {
  if (heads < 0 || heads > 0x7FFFFFFF / kMaxDim) return false;
  if (heads == 0 || T == 0) return true;
  return stride >= (int64_t)heads * D && stride <= INT64_MAX / 4 && product_fits(T, stride * 2);
}

int64_t slots_of(const farn_kv_cache* c) { return c->n_pages * c->page_size; }

// The cache's own numbers and pointers.
bool cache_ok(const farn_kv_cache* c) {
  if (!c || (c->format != FARN_CACHE_FP8 && c->format != FARN_CACHE_NVFP4)) return false;
  if (c->n_pages < 0 || c->page_size < 1 || c->heads < 1 || c->heads > 0x7FFFFFFF / kMaxDim ||
      c->head_dim < 1 || c->head_dim > kMaxDim)
    return false;
  if (c->n_pages > 0x7FFFFFFF || slots_of(c) > 0x7FFFFFFF) return false;    // slots are int32
  if (c->format == FARN_CACHE_NVFP4 &&
      (c->head_dim % 16 != 0 || !isfinite(c->k_tensor_scale) || c->k_tensor_scale <= 0.0f ||
       !isfinite(c->v_tensor_scale) || c->v_tensor_scale <= 0.0f))
    return false;
  if (c->n_pages == 0) return true;
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return false;
  return c->format != FARN_CACHE_FP8 ||
         (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3u) == 0;
}

struct Span {
  const void* at;
  int64_t bytes;
};
void cache_spans(const farn_kv_cache* c, Span s[4]) {
  const int64_t rows = slots_of(c) * c->heads;
  const bool fp8 = c->format == FARN_CACHE_FP8;
  const int64_t codes = rows * (fp8 ? c->head_dim : c->head_dim / 2);
  const int64_t scales = rows * (fp8 ? 4 : c->head_dim / 16);
  s[0] = Span{c->k_codes, codes};
  s[1] = Span{c->v_codes, codes};
  s[2] = Span{c->k_scale, scales};
  s[3] = Span{c->v_scale, scales};
}

void set_cache(Cache* to, const farn_kv_cache* c) {
  to->codes[0] = static_cast<uint8_t*>(c->k_codes);
  to->codes[1] = static_cast<uint8_t*>(c->v_codes);
  to->scale[0] = c->k_scale;
  to->scale[1] = c->v_scale;
  to->g[0] = c->k_tensor_scale;
  to->g[1] = c->v_tensor_scale;
  to->slots = slots_of(c);
}

// for reading, 8 elements at a time, or (write) four
bool cache_aligned(const farn_kv_cache* c, bool write) {
  const uintptr_t need = (c->format == FARN_CACHE_FP8 ? 8u : 4u) / (write ? 2u : 1u) - 1u;
  return (((uintptr_t)c->k_codes | (uintptr_t)c->v_codes) & need) == 0;
}

typedef void (*ReadKernel)(const ReadParams);

template <int FMT>
ReadKernel read_kernel(int lpt) {
  return lpt == 32 ? cache_read_kernel<FMT, 32>
                   : lpt == 16 ? cache_read_kernel<FMT, 16>
                               : lpt == 8 ? cache_read_kernel<FMT, 8> : cache_read_kernel<FMT, 4>;
}

typedef void (*HeadsKernel)(const HeadsParams);

template <int FMT, bool HALF>
HeadsKernel vector_kernel(int D) {
  return D <= 64 ? heads_kernel<8, FMT, HALF>
                 : D <= 128 ? heads_kernel<16, FMT, HALF> : heads_kernel<32, FMT, HALF>;
}
template <int FMT>
HeadsKernel vector_kernel(int D, bool half) {
  return half ? vector_kernel<FMT, true>(D) : vector_kernel<FMT, false>(D);
}

int launch_heads(const farn_ctx* ctx, HeadsParams& p, int fmt, bool cache_vec,
                 cudaStream_t stream) {
  // Two runs of four elements per lane; in halves, the lanes of the rotated part
  // have nothing else, and for NVFP4 they are all there is, four to a block.
  const bool half = !p.interleaved && p.R > 0;
  bool vec = ctx->force_variant != kVariantGeneric && p.D % 8 == 0 && p.D <= 256 && cache_vec &&
             (!half || p.R % 8 == 0) &&
             !(half && fmt == FARN_CACHE_NVFP4 && (p.R != p.D || p.D % 32 != 0));
  auto aligned8 = [](const void* at, int64_t stride) {
    return ((uintptr_t)at & 7u) == 0 && stride % 4 == 0;
  };
  for (int i = 0; i < 3 && vec; ++i)
    if (p.heads[i] && !aligned8(p.in[i], p.in_stride[i])) vec = false;
  for (int i = 0; i < 2 && vec; ++i) {
    if (p.heads[i] && p.weight[i] && !aligned8(p.weight[i], 0)) vec = false;
    if (p.heads[i] && (i == 0 || fmt == 0) && !aligned8(p.out[i], p.out_stride[i])) vec = false;
  }
  HeadsKernel k;
  int64_t tasks;
  if (vec) {
    const int rows = p.D <= 64 ? 4 : p.D <= 128 ? 2 : 1;
    int64_t passes = 0;
    for (int i = 0; i < 3; ++i) passes += (p.heads[i] + rows - 1) / rows;
    // A warp per token for long calls, so that its angles serve all the
    // token's heads; short calls spread a token's heads over more warps.
    const int64_t want = (int64_t)ctx->num_sms * 16;
    int64_t groups = (want + p.T - 1) / p.T;
    p.groups = (int)(groups < 1 ? 1 : groups > passes ? passes : groups);
    tasks = p.T * p.groups;
    k = fmt == 0 ? vector_kernel<0>(p.D, half)
                 : fmt == FARN_CACHE_FP8 ? vector_kernel<FARN_CACHE_FP8>(p.D, half)
                                         : vector_kernel<FARN_CACHE_NVFP4>(p.D, half);
  } else {
    p.groups = 1;
    tasks = p.T * ((int64_t)p.heads[0] + p.heads[1] + p.heads[2]);
    k = fmt == 0 ? heads_plain_kernel<0>
                 : fmt == FARN_CACHE_FP8 ? heads_plain_kernel<FARN_CACHE_FP8>
                                         : heads_plain_kernel<FARN_CACHE_NVFP4>;
  }
  const int warps = vec ? 1 : kWarps;
  int64_t grid = (tasks + warps - 1) / warps;
  const int64_t most = (int64_t)ctx->num_sms * 256 / warps;
  if (grid > most) grid = most;
  return launch(ctx, k, grid, warps * 32, stream, p);
}

// Checks and launch of every form: `cache` NULL for keys in bf16; q NULL and
// rotated false for the plain write.
int run_heads(const farn_ctx* ctx, int64_t T, int D, const void* const in[3], const int heads[3],
              const int64_t in_stride[3], const void* const weight[2], float eps,
              const int32_t* positions, int axes, const int* sections, const float* freqs, int R,
              int interleaved, void* const out[2], const int64_t out_stride[2],
              const farn_kv_cache* cache, const int32_t* slots, cudaStream_t stream) {
  if (!ctx || T < 0 || T > 0x7FFFFFFF || D < 1 || D > kMaxDim || R < 0 || R > D || R % 2 != 0 ||
      !isfinite(eps) || eps < 0.0f)
    return FARN_ERR_INVALID_ARG;
  HeadsParams p;
  memset(&p, 0, sizeof p);
  int64_t all = 0;
  for (int i = 0; i < 3; ++i) {
    if (!heads_size_ok(T, heads[i], D, in_stride[i])) return FARN_ERR_INVALID_ARG;
    all += heads[i];
  }
  if (all < 1 || all > 0x7FFFFFFF) return FARN_ERR_INVALID_ARG;
  if (R > 0) {
    if (axes < 1 || axes > kMaxAxes || !sections) return FARN_ERR_INVALID_ARG;
    int64_t pairs = 0;
    for (int a = 0; a < axes; ++a) {
      if (sections[a] < 0) return FARN_ERR_INVALID_ARG;
      pairs += sections[a];
      if (pairs > R / 2) return FARN_ERR_INVALID_ARG;
      p.axis_end[a] = (int)pairs;
    }
    if (pairs != R / 2) return FARN_ERR_INVALID_ARG;
    for (int a = axes - 1; a < kMaxAxes; ++a) p.axis_end[a] = R;      // the last takes the rest
  }
  if (cache && (!cache_ok(cache) || cache->heads != heads[1] || cache->head_dim != D))
    return FARN_ERR_INVALID_ARG;
  if (T == 0) return FARN_OK;
  for (int i = 0; i < 3; ++i)
    if (heads[i] && (!in[i] || ((uintptr_t)in[i] & 1u))) return FARN_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i) {
    if (!heads[i]) continue;
    if ((uintptr_t)weight[i] & 1u) return FARN_ERR_INVALID_ARG;
    if ((i == 0 || !cache) && (!out[i] || ((uintptr_t)out[i] & 1u) ||
                               !heads_size_ok(T, heads[i], D, out_stride[i])))
      return FARN_ERR_INVALID_ARG;
  }
  if (R > 0 && (!positions || !freqs || ((uintptr_t)positions & 3u) || ((uintptr_t)freqs & 3u)))
    return FARN_ERR_INVALID_ARG;
  if (cache && (!slots || ((uintptr_t)slots & 3u))) return FARN_ERR_INVALID_ARG;

  // What is written may not lie over what is read, but for an output over
  // its own input; nor may two outputs meet.
  Rows ins[3], outs[2];
  for (int i = 0; i < 3; ++i)
    ins[i] = Rows{heads[i] ? in[i] : nullptr, in_stride[i] * 2, (int64_t)heads[i] * D * 2, T};
  for (int i = 0; i < 2; ++i)
    outs[i] = Rows{heads[i] && (i == 0 || !cache) ? out[i] : nullptr, out_stride[i] * 2,
                   (int64_t)heads[i] * D * 2, T};
  const Span reads[5] = {{heads[0] ? weight[0] : nullptr, D * 2},
                         {heads[1] ? weight[1] : nullptr, D * 2},
                         {R ? positions : nullptr, (R ? axes : 0) * T * 4},
                         {R ? freqs : nullptr, R * 2}, {cache ? slots : nullptr, T * 4}};
  for (int o = 0; o < 2; ++o) {
    if (!outs[o].at) continue;
    for (int i = 0; i < 3; ++i)
      if (ins[i].at && !(i == o && same_rows(outs[o], ins[i])) && rows_overlap(outs[o], ins[i]))
        return FARN_ERR_ALIAS;
    for (const Span& r : reads)
      if (r.at && overlaps(outs[o].at, outs[o].span(), r.at, r.bytes)) return FARN_ERR_ALIAS;
  }
  if (outs[0].at && outs[1].at && rows_overlap(outs[0], outs[1])) return FARN_ERR_ALIAS;
  if (cache) {
    Span c[4];
    cache_spans(cache, c);
    for (int a = 0; a < 4; ++a) {
      for (int b = 0; b < a; ++b)
        if (overlaps(c[a].at, c[a].bytes, c[b].at, c[b].bytes)) return FARN_ERR_ALIAS;
      for (int i = 0; i < 3; ++i)
        if (ins[i].at && overlaps(c[a].at, c[a].bytes, ins[i].at, ins[i].span()))
          return FARN_ERR_ALIAS;
      for (const Span& r : reads)
        if (r.at && overlaps(c[a].at, c[a].bytes, r.at, r.bytes)) return FARN_ERR_ALIAS;
      if (outs[0].at && overlaps(c[a].at, c[a].bytes, outs[0].at, outs[0].span()))
        return FARN_ERR_ALIAS;
    }
    set_cache(&p.cache, cache);
  }
  if (ctx->fault_launch) return FARN_ERR_CUDA;
  for (int i = 0; i < 3; ++i) {
    p.in[i] = static_cast<const uint16_t*>(in[i]);
    p.in_stride[i] = in_stride[i];
    p.heads[i] = heads[i];
  }
  for (int i = 0; i < 2; ++i) {
    p.out[i] = static_cast<uint16_t*>(out[i]);
    p.out_stride[i] = out_stride[i];
    p.weight[i] = static_cast<const uint16_t*>(weight[i]);
  }
  p.D = D;
  p.R = R;
  p.interleaved = interleaved != 0;
  p.eps = eps;
  p.positions = positions;
  p.freqs = freqs;
  p.T = T;
  p.slots = slots;
  return launch_heads(ctx, p, cache ? cache->format : 0, !cache || cache_aligned(cache, true),
                      stream);
}

}  // namespace

extern "C" {

int farn_qk_norm_rope(const farn_ctx* ctx, int64_t T, int D, const void* q, int q_heads,
                      int64_t q_stride, const void* k, int k_heads, int64_t k_stride,
                      const void* q_weight, const void* k_weight, float eps,
                      const int32_t* positions, int axes, const int* sections,
                      const float* freqs, int R, int interleaved, void* q_out,
                      int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                      cudaStream_t stream) {
  const void* in[3] = {q, k, nullptr};
  const int heads[3] = {q_heads, k_heads, 0};
  const int64_t in_stride[3] = {q_stride, k_stride, 0};
  const void* weight[2] = {q_weight, k_weight};
  void* out[2] = {q_out, k_out};
  const int64_t out_stride[2] = {q_out_stride, k_out_stride};
  return run_heads(ctx, T, D, in, heads, in_stride, weight, eps, positions, axes, sections, freqs,
                   R, interleaved, out, out_stride, nullptr, nullptr, stream);
}

int farn_qk_norm_rope_cache(const farn_ctx* ctx, int64_t T, int D, const void* q, int q_heads,
                            int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, int kv_heads, const void* q_weight,
                            const void* k_weight, float eps, const int32_t* positions, int axes,
                            const int* sections, const float* freqs, int R, int interleaved,
                            void* q_out, int64_t q_out_stride, const farn_kv_cache* cache,
                            const int32_t* slots, cudaStream_t stream) {
  if (!cache || kv_heads < 1) return FARN_ERR_INVALID_ARG;
  const void* in[3] = {q, k, v};
  const int heads[3] = {q_heads, kv_heads, kv_heads};
  const int64_t in_stride[3] = {q_stride, k_stride, v_stride};
  const void* weight[2] = {q_weight, k_weight};
  void* out[2] = {q_out, nullptr};
  const int64_t out_stride[2] = {q_out_stride, 0};
  return run_heads(ctx, T, D, in, heads, in_stride, weight, eps, positions, axes, sections, freqs,
                   R, interleaved, out, out_stride, cache, slots, stream);
}

int farn_kv_write(const farn_ctx* ctx, int64_t T, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, const farn_kv_cache* cache, const int32_t* slots,
                  cudaStream_t stream) {
  if (!cache || cache->heads < 1) return FARN_ERR_INVALID_ARG;
  const void* in[3] = {nullptr, k, v};
  const int heads[3] = {0, cache->heads, cache->heads};
  const int64_t in_stride[3] = {0, k_stride, v_stride};
  const void* weight[2] = {nullptr, nullptr};
  void* out[2] = {nullptr, nullptr};
  const int64_t out_stride[2] = {0, 0};
  return run_heads(ctx, T, cache->head_dim, in, heads, in_stride, weight, 0.0f, nullptr, 0,
                   nullptr, nullptr, 0, 0, out, out_stride, cache, slots, stream);
}

int farn_kv_read(const farn_ctx* ctx, const farn_kv_cache* cache, const int32_t* table, int B,
                 int64_t width, const int32_t* offsets, int64_t n_tokens, void* k_out,
                 void* v_out, cudaStream_t stream) {
  if (!ctx || !cache_ok(cache) || B < 0 || width < 0 || width > 0x7FFFFFFF || n_tokens < 0 ||
      n_tokens > 0x7FFFFFFF)
    return FARN_ERR_INVALID_ARG;
  const int64_t row = (int64_t)cache->heads * cache->head_dim;
  if (!product_fits(n_tokens, row * 2) || !product_fits(width, (int64_t)B * 4))
    return FARN_ERR_INVALID_ARG;
  if (row >= (1 << 26)) return FARN_ERR_UNSUPPORTED;
  if (n_tokens == 0 || B == 0) return FARN_OK;
  if ((width > 0 && !table) || !offsets || !k_out || !v_out || ((uintptr_t)table & 3u) ||
      ((uintptr_t)offsets & 3u) || ((uintptr_t)k_out & 1u) || ((uintptr_t)v_out & 1u))
    return FARN_ERR_INVALID_ARG;
  const int64_t ob = n_tokens * row * 2;
  Span c[6];
  cache_spans(cache, c);
  c[4] = Span{table, B * width * 4};
  c[5] = Span{offsets, ((int64_t)B + 1) * 4};
  for (const Span& s : c)
    if (overlaps(k_out, ob, s.at, s.bytes) || overlaps(v_out, ob, s.at, s.bytes))
      return FARN_ERR_ALIAS;
  if (overlaps(k_out, ob, v_out, ob)) return FARN_ERR_ALIAS;
  if (ctx->fault_launch) return FARN_ERR_CUDA;
  ReadParams p;
  memset(&p, 0, sizeof p);
  set_cache(&p.cache, cache);
  p.heads = cache->heads;
  p.D = cache->head_dim;
  p.page_size = cache->page_size;
  p.pages = cache->n_pages;
  p.table = table;
  p.B = B;
  p.width = width;
  p.offsets = offsets;
  p.tokens = n_tokens;
  p.out[0] = static_cast<uint16_t*>(k_out);
  p.out[1] = static_cast<uint16_t*>(v_out);
  const bool vec = ctx->force_variant != kVariantGeneric && cache->head_dim % 8 == 0 &&
                   cache_aligned(cache, false) && aligned16(k_out) && aligned16(v_out);
  if (!vec)
    return launch(ctx,
                  cache->format == FARN_CACHE_FP8 ? cache_read_plain_kernel<FARN_CACHE_FP8>
                                                  : cache_read_plain_kernel<FARN_CACHE_NVFP4>,
                  (n_tokens + kPlainTokens - 1) / kPlainTokens, kReadThreads, stream, p);
  const int64_t vecs = row / 8;
  const int lpt = vecs > 16 ? 32 : vecs > 8 ? 16 : vecs > 4 ? 8 : 4;
  const int64_t per = (kReadThreads / 32) * (32 / lpt) * kReadTokens;
  return launch(ctx,
                cache->format == FARN_CACHE_FP8 ? read_kernel<FARN_CACHE_FP8>(lpt)
                                                : read_kernel<FARN_CACHE_NVFP4>(lpt),
                (n_tokens + per - 1) / per, kReadThreads, stream, p);
}

}  // extern "C"

// What the host files of libfarn.so share: the context, the kernel variant
// numbers and small argument helpers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "farn.h"

enum {
  kVariantRow = 0,
  kVariantCluster = 1,
  kVariantGeneric = 2,
  kVariantBulk = 3,
  kVariantStage = 4,
  kVariantCombine = 5,   // the MoE combine's one-CTA-per-row gather kernel
  kVariantTensor = 6,    // the products: tensor cores, one CTA per tile (and part of a row)
  kVariantPair = 7,      // the products: tensor cores, a pair of CTAs per tile
  kVariantAuto = -1
};

struct farn_ctx {
  int device;
  int num_sms;
  int max_cluster;     // largest power-of-two cluster size that can be scheduled
  int force_variant;   // kVariantAuto unless FARN_VARIANT says otherwise
  int force_cluster;   // 0 = choose; else CTAs per row for the cluster variant
  int force_vpt;       // 0 = choose; else 16-byte vectors per thread
  int pdl;             // launch with programmatic stream serialisation
  int64_t small_t;     // below this many rows a call counts as latency bound
  int bulk;            // 1: the TMA-staged kernel serves long inputs by default
  int bulk_ctas;       // resident bulk CTAs per SM (1 or 2)
  int stage;           // 1: the cp.async-staged kernel serves long inputs
  int stage_r;         // 0 = choose; else chunks in flight per thread (8/12/16)
  int stage_ctas;      // 0 = choose; else resident stage CTAs per SM (1..4)
  int64_t stage_min_t; // the stage kernel serves calls with at least this many rows,
  int64_t stage_min_bytes;  // or half as many that read at least this many bytes
  int stage_regs[4][2];  // registers per thread of the staged kernels
                         // [plain, FP8, MoE combine, NVFP4][4 vectors]
  int max_smem;        // opt-in shared memory per CTA, bytes
  int* d_status;       // device status word of the bulk kernel (256 B block)
  int fault_launch;    // FARN_FAULT_INJECT=launch at create: every launch fails
  int stall_test;      // FARN_FAULT_INJECT=stall at create: the TMA-staged kernel's
                       // CTA 0 runs its bounded waits out (a test of the status word)
  int tc_tile;         // 0 = choose; else the products' tiles: 64 slots by one CTA, or 256
                       // (NVFP4: 224) by a pair
  int tc_split;        // 0 = choose; else CTAs that split a row: 1, 2 or 4
  int route_ok;        // the router's kernels are set up
  void* encode_tiled;  // the driver's tensor-map encoder; null: the products' tensor-core
                       // kernels are not set up, and the plain one takes every call
  int max_clusters[3]; // clusters of 1, 2 and 4 of their CTAs that fit the device at a time
};

namespace farn_host {

// One-time kernel set-up on the current device (farn_create).  False: the
// router, or the products' tensor-core kernels, cannot be had.
bool route_setup(const farn_ctx* ctx);
bool product_setup(farn_ctx* ctx);

inline bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  if (na <= 0 || nb <= 0) return false;
  uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// True for sizes (counts of bytes or elements) whose product fits an int64.
inline bool product_fits(int64_t a, int64_t b) {
  return a == 0 || b == 0 || a <= INT64_MAX / b;
}

struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
    if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

}  // namespace farn_host

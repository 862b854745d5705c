// Plan queries of the FP8 and NVFP4 products against a context made up on the
// host: no device is needed.
//   product_plan_probe fp8|nvfp4 T N H
//   product_plan_probe experts SLOTS E N H     (FP8, gathered rows, a workspace given)
// prints the status, the variant and the CTAs per tile; experts: and the
// workspace's bytes.
#include <cuda_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "farn_internal.h"

int main(int argc, char** argv) {
  if (argc < 5) return 2;
  farn_ctx c;
  memset(&c, 0, sizeof c);
  c.force_variant = kVariantAuto;
  c.num_sms = 152;
  c.max_clusters[0] = 152;
  c.max_clusters[1] = 76;
  c.max_clusters[2] = 36;
  c.max_smem = 227 * 1024;
  c.encode_tiled = &c;          // only its presence matters to a plan
  c.fp8_ok = 1;
  void* at[6];
  for (int i = 0; i < 6; ++i) at[i] = (void*)((uintptr_t)(i + 1) << 40);
  long long v[4] = {};
  for (int i = 0; i + 2 < argc && i < 4; ++i) v[i] = atoll(argv[i + 2]);
  int variant = -1, ctas = -1, threads = -1, st;
  int64_t bytes = 0;
  if (!strcmp(argv[1], "fp8")) {
    st = farn_plan_fp8_matmul(&c, at[0], at[1], v[0], v[1], v[2], at[2], &variant, &ctas, &threads);
  } else if (!strcmp(argv[1], "nvfp4")) {
    st = farn_plan_nvfp4_matmul(&c, at[0], at[1], at[2], at[3], v[0], v[1], v[2], at[4], &variant,
                                &ctas, &threads);
  } else {
    if (argc != 6) return 2;
    st = farn_plan_fp8_grouped_matmul(&c, at[0], v[0], (const int32_t*)at[1], v[0], at[2],
                                      (int)v[1], v[2], v[3], at[3], at[4], &variant, &ctas,
                                      &threads);
    if (farn_fp8_grouped_workspace(&c, v[0], (int)v[1], v[2], v[3], &bytes) != FARN_OK) return 3;
  }
  printf("%d %d %d %lld\n", st, variant, ctas, (long long)bytes);
  return 0;
}

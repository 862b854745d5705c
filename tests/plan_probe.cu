// Plan queries against a context made up on the host: no device is needed.
//   plan_probe SMS CLUSTERS1 CLUSTERS2 CLUSTERS4 SPLIT SLOTS E N H
// prints the status, the variant and the CTAs per tile of a grouped product.
#include <cuda_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "farn_internal.h"

int main(int argc, char** argv) {
  if (argc != 10) return 2;
  farn_ctx c;
  memset(&c, 0, sizeof c);
  c.force_variant = kVariantAuto;
  c.num_sms = atoi(argv[1]);
  for (int i = 0; i < 3; ++i) c.max_clusters[i] = atoi(argv[2 + i]);
  c.tc_split = atoi(argv[5]);
  c.max_smem = 227 * 1024;
  c.encode_tiled = &c;          // only its presence matters to a plan
  const long long S = atoll(argv[6]), N = atoll(argv[8]), H = atoll(argv[9]);
  void* at[3];
  for (int i = 0; i < 3; ++i) at[i] = (void*)((uintptr_t)(i + 1) << 32);
  int variant = -1, ctas = -1, threads = -1;
  const int st = farn_plan_grouped_matmul(&c, at[0], S, nullptr, S, at[1], atoi(argv[7]), N, H,
                                          at[2], &variant, &ctas, &threads);
  printf("%d %d %d\n", st, variant, ctas);
  return 0;
}

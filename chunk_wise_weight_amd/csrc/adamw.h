// The AdamW step over many tensors (kernels_adamw.hip): the tensors of one launch, in its arguments.
#pragma once

#include "common.h"

// Up to kAdamTable tensors, cut into chunks of kAdamChunk elements (the last
// one of each shorter). As a kernel argument the table needs no device copy;
// it stays within the 4 KiB that every launch may pass.
constexpr int kAdamTable = 60, kAdamChunk = 4096, kAdamBlock = 256;
struct AdamTable {
  void *w[kAdamTable], *m[kAdamTable], *v[kAdamTable];
  const void *g[kAdamTable];
  bf16_t *copy[kAdamTable];        // nullable
  int16_t *top[kAdamTable];        // 8-bit states: [2][blocks]
  uint32_t first[kAdamTable + 1];  // chunks before tensor i
  uint32_t tail[kAdamTable];       // elements of its last chunk
  uint8_t w_f32[kAdamTable], g_f32[kAdamTable];
  int n;
  int tensor0;  // number in the call's list of tensor 0
};

struct AdamArgs {
  double beta1, beta2, eps, lr, decay, tau;
  double log1, log2;  // of the betas
  long long step;
  const long long *step_dev;
  const float *lr_dev;
  const float *norm;  // nullable
  uint32_t seed;
};

hipError_t launch_adamw(const AdamTable &t, const AdamArgs &a, bool bits8, hipStream_t s);
// values of codes: out[i] (in w) from codes m[i] or v[i] (in m) by tops row `second`
hipError_t launch_adamw_values(const AdamTable &t, bool second, hipStream_t s);

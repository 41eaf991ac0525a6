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

// What all elements of a step share.
struct AdamStep {
  float lr1, root2;  // lr / (1 - b1^t), (1 - b2^t)^-1/2
  float shrink;      // lr decay
  uint32_t key;      // of the random bits, from seed and step
};
// A beta in two fp32 parts, so that it and `rest` = 1 - beta add up to one: rounded to one part, a beta2 of 0.9999 is off
// by U / 4 of every moment it meets and by 10^-4 of what it leaves to the gradient (U = 2^-24).
struct AdamDecay {
  float hi, lo, rest;
};
inline AdamDecay adam_decay(double b) {
  const float hi = (float)b;
  return {hi, (float)(b - (double)hi), (float)(1.0 - b)};
}
struct AdamArgs {
  AdamDecay decay1, decay2;  // fp32 moments
  double beta1, beta2, lr, decay, tau;
  double log1, log2;  // of the betas
  float eps;
  AdamStep fixed;  // where neither of the next two is given
  const long long *step_dev;
  const float *lr_dev;
  long long step;
  const float *norm;  // nullable
  uint32_t seed;
};

static_assert(sizeof(AdamTable) + sizeof(AdamArgs) <= 4096, "every launch may pass 4 KiB of arguments");

// The random bits' mixing: two rounds of a shift and a multiplication by an odd
// constant, which reach every bit of the result.
__host__ __device__ inline uint32_t adam_mix(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x6C8E9CF5u;
  h = (h ^ (h >> 13)) * 0x51ED2701u;
  return h ^ (h >> 16);
}
constexpr uint32_t kGolden = 0x9E3779B1u;  // 2^32 by the golden ratio, odd
__host__ __device__ inline uint32_t adam_key(uint32_t seed, long long step) {
  return adam_mix(seed + kGolden * adam_mix((uint32_t)step));
}

// stream: the arrays are more than the caches hold
hipError_t launch_adamw(const AdamTable &t, const AdamArgs &a, bool bits8, bool stream, hipStream_t s);
// values of codes: out[i] (in w) from codes m[i] or v[i] (in m) by tops row `second`
hipError_t launch_adamw_values(const AdamTable &t, bool second, bool stream, hipStream_t s);

// The gradient-norm kernels (kernels_grads.hip): the tensors of one launch, in its arguments.
#pragma once

#include "common.h"

// Up to kGradTable tensors, cut into chunks of kGradBytes (the last one of
// each tensor shorter). As a kernel argument it needs no device copy, so
// a call reads nothing that could change or be freed behind it; 152 of them
// stay within the 4 KiB that every launch may pass.
constexpr int kGradTable = 152, kGradBytes = 16384;
struct GradTable {
  const void *g[kGradTable];
  void *out[kGradTable];
  uint32_t first[kGradTable + 1];  // chunks before tensor i
  uint32_t tail[kGradTable];       // elements of its last chunk
  uint8_t f32[kGradTable];
  int n;
};

// What gradients are multiplied by, mantissa * 2^exponent.
struct GradFactor {
  float mantissa;
  int exponent;
};

// Workgroups of all norm launches of a call together (besides one per further table): one partial sum each.
constexpr int kGradGroups = 2048;

// part[blockIdx.x] = sum of squares of its chunks. stream: the gradients are more than the caches hold.
hipError_t launch_grad_squares(const GradTable &t, double *part, int groups, bool stream, hipStream_t s);
// *norm = sqrt(sum of part[0 .. n)); *factor (nullable) = min(1, tau / norm), 1 where the norm is not finite
hipError_t launch_grad_norm(const double *part, int n, float tau, float *norm, GradFactor *factor, hipStream_t s);
// out = g * *factor
hipError_t launch_grad_scale(const GradTable &t, const GradFactor *factor, bool stream, hipStream_t s);

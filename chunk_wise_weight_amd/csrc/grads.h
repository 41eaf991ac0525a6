// The gradient-norm kernels (kernels_grads.hip): the tensors of one launch, in its arguments.
#pragma once

#include "common.h"

// Up to kGradTable tensors, cut into chunks of `chunk` elements (the last one
// of each tensor shorter). As a kernel argument it needs no device copy, so a
// call reads nothing that could change or be freed behind it; 152 of them stay
// within the 4 KiB that every launch may pass.
constexpr int kGradTable = 152;
struct GradTable {
  const void *g[kGradTable];
  void *out[kGradTable];
  uint32_t first[kGradTable + 1];  // chunks before tensor i
  uint32_t tail[kGradTable];       // elements of its last chunk
  uint8_t f32[kGradTable];
  int n;
  uint32_t chunk;
};

// Workgroups of all norm launches of a call together (besides one per further table): one partial sum each.
constexpr int kGradGroups = 2048;

// part[blockIdx.x] = sum of squares of its chunks
hipError_t launch_grad_squares(const GradTable &t, double *part, int groups, hipStream_t s);
// *norm = sqrt(sum of part[0 .. n))
hipError_t launch_grad_norm(const double *part, int n, float *norm, hipStream_t s);
// out = g * min(1, tau / norm) (g as it is where the norm is not finite); norm (nullable) receives the norm
hipError_t launch_grad_scale(const GradTable &t, const double *part, int n, float tau, float *norm, int groups,
                             hipStream_t s);

// Grids of many workgroups.
#pragma once

#include <hip/hip_runtime.h>

// A launch of one workgroup per row or more: threads of a grid's side are
// counted in 32 bits, so many rows take a second side. group_index() is the
// workgroup's number; the last ones may lie past `groups`.
constexpr long long kGridSide = 1 << 20;
inline dim3 group_grid(long long groups) {
  if (groups <= kGridSide) return dim3((unsigned)groups);
  return dim3((unsigned)kGridSide, (unsigned)((groups + kGridSide - 1) / kGridSide));
}
__device__ __forceinline__ long long group_index() { return (long long)blockIdx.y * gridDim.x + blockIdx.x; }

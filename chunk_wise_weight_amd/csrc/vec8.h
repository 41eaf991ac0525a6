// W consecutive elements of a row as fp32, for the row-wise kernels: eight,
// moved in 16-byte accesses, or one.
//
// Eight elements may start at any of them: gfx950 reads and writes global
// memory at any byte address, so a row that starts on an odd element costs a
// second cache line now and then and no other code. `on` false reads zeros and
// writes nothing.
#pragma once

#include "common.h"

struct Raw8b {
  uint32_t u[4];
};
struct Raw8f {
  float f[8];
};

__device__ __forceinline__ void load_w(const bf16_t *p, bool on, float (&v)[8]) {
  Raw8b r = {{0, 0, 0, 0}};
  if (on) __builtin_memcpy(&r, p, 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(r.u[j] << 16);
    v[2 * j + 1] = __uint_as_float(r.u[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load_w(const float *p, bool on, float (&v)[8]) {
  Raw8f r = {{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}};
  if (on) __builtin_memcpy(&r, p, 32);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = r.f[j];
}
__device__ __forceinline__ void load_w(const bf16_t *p, bool on, float (&v)[1]) { v[0] = on ? bf16_to_f32(*p) : 0.f; }
__device__ __forceinline__ void load_w(const float *p, bool on, float (&v)[1]) { v[0] = on ? *p : 0.f; }

__device__ __forceinline__ void store_w(bf16_t *p, bool on, const float (&v)[8]) {
  Raw8b r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r.u[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  if (on) __builtin_memcpy(p, &r, 16);
}
__device__ __forceinline__ void store_w(float *p, bool on, const float (&v)[8]) {
  Raw8f r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r.f[j] = v[j];
  if (on) __builtin_memcpy(p, &r, 32);
}
__device__ __forceinline__ void store_w(bf16_t *p, bool on, const float (&v)[1]) {
  if (on) *p = f32_to_bf16(v[0]);
}
__device__ __forceinline__ void store_w(float *p, bool on, const float (&v)[1]) {
  if (on) *p = v[0];
}

// The same of a parameter that is fp32 or bf16 as the caller has it (a branch
// all threads take alike); a NULL parameter reads as ones.
template <int W>
__device__ __forceinline__ void load_param(const void *p, int f32, long long at, bool on, float (&v)[W]) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = 1.f;
  } else if (f32) {
    load_w(reinterpret_cast<const float *>(p) + at, on, v);
  } else {
    load_w(reinterpret_cast<const bf16_t *>(p) + at, on, v);
  }
}

// W consecutive elements of a row as fp32, for the row-wise kernels: eight,
// moved in 16-byte accesses, or one.
//
// Eight elements may start at any of them: gfx950 reads and writes global
// memory at any byte address, so a row that starts on an odd element costs a
// second cache line now and then and no other code. `on` false reads zeros and
// writes nothing.
#pragma once

#include "common.h"
#include "grid.h"

// Eight elements as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  uint32_t u[4];
};
template <>
struct Raw8<float> {
  float f[8];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T *p, bool on) {
  Raw8<T> r = {};
  if (on) __builtin_memcpy(&r, p, sizeof r);
  return r;
}
__device__ __forceinline__ void expand(const Raw8<bf16_t> &r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(r.u[j] << 16);
    v[2 * j + 1] = __uint_as_float(r.u[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void expand(const Raw8<float> &r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = r.f[j];
}

template <typename T>
__device__ __forceinline__ void load_w(const T *p, bool on, float (&v)[8]) {
  expand(load_raw(p, on), v);
}
__device__ __forceinline__ void load_w(const bf16_t *p, bool on, float (&v)[1]) { v[0] = on ? bf16_to_f32(*p) : 0.f; }
__device__ __forceinline__ void load_w(const float *p, bool on, float (&v)[1]) { v[0] = on ? *p : 0.f; }

__device__ __forceinline__ void store_w(bf16_t *p, bool on, const float (&v)[8]) {
  Raw8<bf16_t> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r.u[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  if (on) __builtin_memcpy(p, &r, 16);
}
__device__ __forceinline__ void store_w(float *p, bool on, const float (&v)[8]) {
  Raw8<float> r;
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

// Behind a kernel's last wide store: the store reads its data registers after
// it issues, and two wait states must pass before an instruction writes one of
// them. No instruction follows at the kernel's end, but in the listing, which
// is checked for this hazard line by line, the code of another branch may.
__device__ __forceinline__ void end_of_stores() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 1");
  __builtin_amdgcn_sched_barrier(0);
}

// Eight elements past the caches' keeping (the `nt` bit), for arrays too large
// for the next kernel to find them there.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void stream_w(bf16_t *p, bool on, const float (&v)[8]) {
  const u32x4_any r = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7])};
  if (on) __builtin_nontemporal_store(r, reinterpret_cast<u32x4_any *>(p));
}

// Eight columns of a row as two runs of four, at p and `gap` elements behind
// (half a row): the fp32 runs of neighbouring threads then lie side by side,
// and each access of a wave covers whole cache lines.
__device__ __forceinline__ Raw8<bf16_t> load_halves(const bf16_t *p, int gap, bool on) {
  Raw8<bf16_t> r = {};
  if (on) {
    __builtin_memcpy(r.u, p, 8);
    __builtin_memcpy(r.u + 2, p + gap, 8);
  }
  return r;
}
__device__ __forceinline__ Raw8<float> load_halves(const float *p, int gap, bool on) {
  Raw8<float> r = {};
  if (on) {
    __builtin_memcpy(r.f, p, 16);
    __builtin_memcpy(r.f + 4, p + gap, 16);
  }
  return r;
}
template <bool STREAM>
__device__ __forceinline__ void store_halves(float *p, int gap, const float (&v)[8]) {
  const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
  typedef f32x4 __attribute__((aligned(4))) any;
  if (STREAM) {
    __builtin_nontemporal_store(a, reinterpret_cast<any *>(p));
    __builtin_nontemporal_store(b, reinterpret_cast<any *>(p + gap));
  } else {
    *reinterpret_cast<any *>(p) = a;
    *reinterpret_cast<any *>(p + gap) = b;
  }
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

// What becomes of a product's sums: bias, activation, residual, and the stores.
#pragma once

#include "act.h"
#include "linear.h"
#include "vec8.h"

__device__ __forceinline__ int clamp8(long long n) { return n < 0 ? 0 : n > 8 ? 8 : (int)n; }

template <int W>
__device__ __forceinline__ void get(const float *p, int n, float (&v)[W]) {
  if (n >= W) {
    __builtin_memcpy(v, p, W * 4);
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = i < n ? p[i] : 0.f;
}
template <int W>
__device__ __forceinline__ void get(const bf16_t *p, int n, float (&v)[W]) {
  if (n >= W) {
    uint32_t u[W / 2];
    __builtin_memcpy(u, p, W * 2);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = i < n ? bf16_to_f32(p[i]) : 0.f;
}
template <int W>
__device__ __forceinline__ void put(float *p, int n, const float (&v)[W]) {
  if (n >= W) {
    __builtin_memcpy(p, v, W * 4);
    end_of_stores();  // the code of the other branch may follow
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < n) p[i] = v[i];
}
template <int W>
__device__ __forceinline__ void put(bf16_t *p, int n, const float (&v)[W]) {
  if (n >= W) {
    uint32_t u[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    __builtin_memcpy(p, u, W * 2);
    end_of_stores();
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < n) p[i] = f32_to_bf16(v[i]);
}

// The same, past the caches' keeping where eight are there: the tiles of a large
// product are written while others still read their operands (the pair of 32768
// x 2560 x 9728 with g and u kept: 2859 -> 2627 us).
template <typename T, int W>
__device__ __forceinline__ void put_past(T *p, int n, const float (&v)[W]) {
  if constexpr (W == 8) {
    if (n >= 8) {
      if constexpr (sizeof(T) == 2) {
        stream_w(p, true, v);
      } else {
        typedef f32x4 any __attribute__((aligned(4)));
        __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<any *>(p));
        __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<any *>(p + 4));
      }
      end_of_stores();
      return;
    }
  }
  put(p, n, v);
}
template <bool NT, typename T, int W>
__device__ __forceinline__ void put_out(T *p, int n, const float (&v)[W]) {
  if constexpr (NT)
    put_past(p, n, v);
  else
    put(p, n, v);
}

// n of 8 elements, the rest zero
template <typename T>
__device__ __forceinline__ Raw8<T> load_some(const T *p, int n) {
  Raw8<T> r = {};
  if (n >= 8) {
    __builtin_memcpy(&r, p, sizeof r);
  } else if (n > 0) {
    T v[8] = {};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) v[i] = p[i];
    __builtin_memcpy(&r, v, sizeof r);
  }
  return r;
}

// n of the W elements from (i, j) on are there. old: the residual's eight, loaded before.
template <typename T, typename O, bool NT = false, int W>
__device__ __forceinline__ void finish(const GemmArgs &g, int z, long long i, long long j, int n, float (&v)[W],
                                       const Raw8<O> *old = nullptr) {
  const long long at = j * g.ldo + i;
  float w[W];
  if (g.bias[0]) {
    get(reinterpret_cast<const T *>(g.bias[0]) + i, n, w);
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] += w[e];
  }
  if (g.pre[0]) put_out<NT>(reinterpret_cast<T *>(g.pre[0]) + at, n, v);
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] = g.scale * act_of(v[e], g.act);
  if (g.res[z]) {
    if constexpr (W == 8) {
      if (old)
        expand(*old, w);
      else
        get(reinterpret_cast<const O *>(g.res[z]) + at, n, w);
    } else {
      get(reinterpret_cast<const O *>(g.res[z]) + at, n, w);
    }
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] += w[e];
  }
  put_out<NT>(reinterpret_cast<O *>(g.out[z]) + at, n, v);
}
// the gated pair: a the gate's products, u the other's
template <typename T, bool NT = false, int W>
__device__ __forceinline__ void finish_pair(const GemmArgs &g, long long i, long long j, int n, float (&a)[W],
                                            float (&u)[W]) {
  const long long at = j * g.ldo + i;
  float w[W];
  if (g.bias[0]) {
    get(reinterpret_cast<const T *>(g.bias[0]) + i, n, w);
#pragma unroll
    for (int e = 0; e < W; ++e) a[e] += w[e];
    get(reinterpret_cast<const T *>(g.bias[1]) + i, n, w);
#pragma unroll
    for (int e = 0; e < W; ++e) u[e] += w[e];
  }
  if (g.pre[0]) {
    put_out<NT>(reinterpret_cast<T *>(g.pre[0]) + at, n, a);
    put_out<NT>(reinterpret_cast<T *>(g.pre[1]) + at, n, u);
  }
#pragma unroll
  for (int e = 0; e < W; ++e) w[e] = act_of(a[e], g.act) * u[e];
  put_out<NT>(reinterpret_cast<T *>(g.out[0]) + at, n, w);
}

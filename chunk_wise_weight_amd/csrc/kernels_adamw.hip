// AdamW over many tensors in one pass, with moments in fp32 or in 8 bits:
//
//   g' = g min(1, tau / N),  m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2
//   w' = w (1 - lr decay) - lr (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps)
//
// 8-bit moments: a block of 256 elements has a top T, the smallest multiple of
// 2^20 that no |x| of the block passes as an fp32 bit pattern (its exponent
// and 3 mantissa bits), in units of 2^20. Code c > 0 stands for the pattern
// (T - most + c) << 20 (0 where that is not positive), most = 127 for m, whose
// sign is the code's top bit, and 255 for v; code 0 stands for 0. So a block
// holds 16 octaves below its largest |m| and 32 below its largest v, with a
// step of 1/8 to 1/16, and both directions are shifts. |x| goes to one of its
// two neighbours at random so that its expectation is kept: rounded to the
// nearest, a second moment would never move, because one step of the recurrence
// changes it by 1 - b2 (10^-3) and a step of the code by 6 to 12 10^-2. A
// second moment that is not zero is not held as zero, because the weight's
// step divides by its root.
//
// The moments of the 8-bit form are computed in fp64 and rounded to fp32 once
// before they become codes. fp32 sums would do for the moments, but not for a
// value next to the border between two codes: there the order of the roundings
// would decide a code, and the same step computed elsewhere (a replica, a
// resumed run on other software) would drift apart. The pass is bound by
// memory either way.
#include "adamw.h"
#include "vec8.h"

namespace {

constexpr int kThreads = 256, kWaveSteps = kAdamChunk / kAdamBlock / (kThreads / 64);

// Four elements as they lie in memory, at any of them; past the caches' keeping with NT.
typedef uint32_t u32x4_el __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_el __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_el __attribute__((aligned(1)));

template <bool NT, typename V>
__device__ __forceinline__ V fetch(const void *p) {
  const V *q = reinterpret_cast<const V *>(p);
  return NT ? __builtin_nontemporal_load(q) : *q;
}
template <bool NT, typename V>
__device__ __forceinline__ void keep(void *p, V v) {
  V *q = reinterpret_cast<V *>(p);
  if (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

// Four elements of a tensor that is fp32 or bf16 (a branch all threads take alike), n of them there.
struct Four {
  uint32_t u[4];
};
template <bool NT>
__device__ __forceinline__ Four get(const void *p, int f32, long long at, int n) {
  Four r = {};
  if (f32) {
    const float *q = reinterpret_cast<const float *>(p) + at;
    if (n >= 4) {
      const u32x4_el v = fetch<NT, u32x4_el>(q);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.u[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) r.u[i] = __float_as_uint(q[i]);
    }
  } else {
    const bf16_t *q = reinterpret_cast<const bf16_t *>(p) + at;
    if (n >= 4) {
      const u32x2_el v = fetch<NT, u32x2_el>(q);
      r.u[0] = v[0];
      r.u[1] = v[1];
    } else {
      uint32_t e[3] = {};
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) e[i] = q[i];
      r.u[0] = e[0] | e[1] << 16;
      r.u[1] = e[2];
    }
  }
  return r;
}
__device__ __forceinline__ void expand(const Four &r, int f32, float (&v)[4]) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.u[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(r.u[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.u[i] & 0xffff0000u);
    }
  }
}
template <bool NT>
__device__ __forceinline__ void put(void *p, int f32, long long at, int n, const float (&v)[4]) {
  if (f32) {
    float *q = reinterpret_cast<float *>(p) + at;
    if (n >= 4) {
      keep<NT>(q, u32x4_el{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
      end_of_stores();
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) q[i] = v[i];
    }
  } else {
    bf16_t *q = reinterpret_cast<bf16_t *>(p) + at;
    if (n >= 4) {
      keep<NT>(q, u32x2_el{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) q[i] = f32_to_bf16(v[i]);
    }
  }
}
// four codes, the first in the low byte
template <bool NT>
__device__ __forceinline__ uint32_t get_codes(const uint8_t *p, int n) {
  if (n >= 4) return fetch<NT, u32_el>(p);
  uint32_t u = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < n) u |= (uint32_t)p[i] << (8 * i);
  return u;
}
template <bool NT>
__device__ __forceinline__ void put_codes(uint8_t *p, int n, uint32_t u) {
  if (n >= 4) {
    keep<NT, u32_el>(p, u);
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < n) p[i] = (uint8_t)(u >> (8 * i));
}

// The value of the low byte of c under a block's top, lowest = top - most.
template <int MOST>
__device__ __forceinline__ float decode(uint32_t c, int lowest) {
  const int code = (int)(c & MOST), k = max(lowest + code, 0);
  const uint32_t u = code ? (uint32_t)k << 20 : 0u;
  return __uint_as_float(MOST == 127 ? u | (c & 128u) << 24 : u);
}

constexpr uint32_t kQuietNan = 0x7FC00000u;  // every NaN's pattern here, so that tops stay below 2^11

__device__ __forceinline__ uint32_t magnitude(float x) { return min(__float_as_uint(x) & 0x7fffffffu, kQuietNan); }

// The code of x of magnitude mag under a block's lowest = top - most, with 16 random bits r.
template <int MOST>
__device__ __forceinline__ uint32_t encode(float x, uint32_t mag, int lowest, uint32_t r) {
  int c = (int)((mag + (r << 4)) >> 20) - lowest;
  if (MOST == 127) {
    if (__any(c < 1)) {  // below the block's smallest value, which few are
      const float least = __uint_as_float(lowest > -1 ? (uint32_t)(lowest + 1) << 20 : 0u);
      const int low = __uint_as_float(mag) >= ((float)r + 0.5f) * 0x1p-16f * least;
      c = c < 1 ? low : c;
    }
  } else {
    c = max(c, 1);
  }
  c = mag ? c : 0;
  return MOST == 127 && c ? (uint32_t)c | (__float_as_uint(x) >> 24 & 128u) : (uint32_t)c;
}

// The largest of a wave's values, in every lane: by rotations within the rows of 16 lanes, then between rows.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, true));  // row_ror:8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, true));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}

__device__ __forceinline__ AdamStep step_of(const AdamArgs &a) {
  if (!a.step_dev && !a.lr_dev) return a.fixed;
  AdamStep s;
  const long long t = a.step_dev ? *a.step_dev : a.step;
  const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
  // 1 - b^t without its cancellation
  const double c1 = -expm1((double)t * a.log1), c2 = -expm1((double)t * a.log2);
  s.lr1 = (float)(lr / c1);
  s.root2 = (float)(1.0 / sqrt(c2));
  s.shrink = (float)(lr * a.decay);
  s.key = adam_key(a.seed, t);
  return s;
}

// sqrt(v) by the hardware's root (1 ulp), with `small` also of the denormals, which it may take as 0: their roots are
// below 2^-63, which is nothing beside an eps of 10^-10.
__device__ __forceinline__ float root(float v, bool small) {
  if (!small) return __builtin_amdgcn_sqrtf(v);
  const bool tiny = v < 0x1p-96f;
  return __builtin_amdgcn_sqrtf(tiny ? v * 0x1p64f : v) * (tiny ? 0x1p-32f : 1.f);
}

// A chunk's tensor, its first element and its elements. One chunk per workgroup.
struct Place {
  int i, n;
  long long at;
};
__device__ __forceinline__ bool place_of(const AdamTable &t, Place &p) {
  const long long c = group_index();
  if (c >= t.first[t.n]) return false;
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  p.i = lo;
  p.at = (c - t.first[lo]) * kAdamChunk;
  p.n = c + 1 == t.first[lo + 1] ? (int)t.tail[lo] : kAdamChunk;
  return true;
}

// FULL: every element of the chunk is there.
template <bool BITS8, bool NT, bool FULL>
__device__ __forceinline__ void step_chunk(const AdamTable &t, const AdamArgs &a, const Place &p) {
  const int i = p.i, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int w_f32 = t.w_f32[i], g_f32 = t.g_f32[i];
  const long long at0 = p.at + wave * kAdamBlock + lane * 4;
  const int left0 = FULL ? kAdamChunk : p.n - wave * kAdamBlock - lane * 4;
  constexpr int SKIP = kThreads / 64 * kAdamBlock;  // from a wave's block to its next
  // everything is loaded before anything is stored
  Four w[kWaveSteps], g[kWaveSteps], m[kWaveSteps], v[kWaveSteps];
  int top[kWaveSteps][2];
  long long blocks = 0;
  if (BITS8) blocks = (long long)(t.first[i + 1] - t.first[i] - 1) * (kAdamChunk / kAdamBlock) +
                      (t.tail[i] + kAdamBlock - 1) / kAdamBlock;
#pragma unroll
  for (int k = 0; k < kWaveSteps; ++k) {
    const long long at = at0 + k * SKIP;
    const int left = FULL ? 4 : left0 - k * SKIP;
    w[k] = get<NT>(t.w[i], w_f32, at, left);
    g[k] = get<NT>(t.g[i], g_f32, at, left);
    if constexpr (BITS8) {
      m[k].u[0] = get_codes<NT>((const uint8_t *)t.m[i] + at, left);
      v[k].u[0] = get_codes<NT>((const uint8_t *)t.v[i] + at, left);
      const long long block = (p.at + wave * kAdamBlock + k * SKIP) / kAdamBlock;
      const bool there = FULL || wave * kAdamBlock + k * SKIP < p.n;
      top[k][0] = there ? t.top[i][block] : 0;
      top[k][1] = there ? t.top[i][blocks + block] : 0;
    } else {
      m[k] = get<NT>(t.m[i], 1, at, left);
      v[k] = get<NT>(t.v[i], 1, at, left);
    }
  }
  const AdamStep s = step_of(a);
  const double b1 = a.beta1, b2 = a.beta2;
  double factor = 1.0;  // of the gradients
  bool clipped = false;
  if (a.norm) {
    const double n = (double)*a.norm;
    clipped = n > a.tau && n <= 3.4028234663852886e38;  // a norm that is not finite clips nothing
    if (clipped) factor = a.tau / n;
  }
  // fp64 holds the factor's square with the betas; fp32 takes it to the gradient first
  const double o1 = (1.0 - b1) * factor, o2 = (1.0 - b2) * factor * factor;
  const float b1f = (float)b1, b2f = (float)b2, o1f = (float)(1.0 - b1), o2f = (float)(1.0 - b2);
  const bool small = a.eps < 1e-10f;
  const uint32_t key = BITS8 ? adam_mix(s.key + kGolden * (uint32_t)(t.tensor0 + i + 1)) : 0u;
#pragma unroll
  for (int k = 0; k < kWaveSteps; ++k) {
    if (!FULL && wave * kAdamBlock + k * SKIP >= p.n) break;  // the wave's block is there, or none of it
    const long long at = at0 + k * SKIP;
    const int left = FULL ? 4 : left0 - k * SKIP;
    float x[4], mk[4], vk[4], wk[4];
    expand(g[k], g_f32, x);
    expand(w[k], w_f32, wk);
    if constexpr (BITS8) {
      uint32_t mm = 0, mv = 0, am[4], av[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const double d = (double)x[e];
        mk[e] = (float)(b1 * (double)decode<127>(m[k].u[0] >> (8 * e), top[k][0] - 127) + o1 * d);
        vk[e] = (float)(b2 * (double)decode<255>(v[k].u[0] >> (8 * e), top[k][1] - 255) + o2 * d * d);
        am[e] = magnitude(mk[e]);
        av[e] = magnitude(vk[e]);
        mm = max(mm, am[e]);
        mv = max(mv, av[e]);
      }
      const int um = (int)((wave_max(mm) + 0xFFFFFu) >> 20), uv = (int)((wave_max(mv) + 0xFFFFFu) >> 20);
      const long long block = (p.at + wave * kAdamBlock + k * SKIP) / kAdamBlock;
      if (lane == 0) {
        t.top[i][block] = (int16_t)um;
        t.top[i][blocks + block] = (int16_t)uv;
      }
      uint32_t nm = 0, nv = 0;
      const uint32_t place = key + (uint32_t)at * kGolden;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t r = adam_mix(place + e * kGolden);
        nm |= encode<127>(mk[e], am[e], um - 127, r & 0xFFFFu) << (8 * e);
        nv |= encode<255>(vk[e], av[e], uv - 255, r >> 16) << (8 * e);
      }
      put_codes<NT>((uint8_t *)t.m[i] + at, left, nm);
      put_codes<NT>((uint8_t *)t.v[i] + at, left, nv);
    } else {
      expand(m[k], 1, mk);
      expand(v[k], 1, vk);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float d = clipped ? (float)((double)x[e] * factor) : x[e];
        mk[e] = fmaf(b1f, mk[e], o1f * d);
        vk[e] = fmaf(b2f, vk[e], o2f * d * d);
      }
      put<NT>(t.m[i], 1, at, left, mk);
      put<NT>(t.v[i], 1, at, left, vk);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float q = s.lr1 * mk[e] * __builtin_amdgcn_rcpf(fmaf(root(vk[e], small), s.root2, a.eps));
      wk[e] = fmaf(-s.shrink, wk[e], wk[e]) - q;
    }
    put<NT>(t.w[i], w_f32, at, left, wk);
    if (t.copy[i]) put<NT>(t.copy[i], 0, at, left, wk);
  }
  end_of_stores();
}

template <bool BITS8, bool NT>
__global__ __launch_bounds__(kThreads) void k_adamw(AdamTable t, AdamArgs a) {
  Place p;
  if (!place_of(t, p)) return;
  if (p.n == kAdamChunk)
    step_chunk<BITS8, NT, true>(t, a, p);
  else
    step_chunk<BITS8, NT, false>(t, a, p);
}

template <bool SECOND, bool NT>
__global__ __launch_bounds__(kThreads) void k_values(AdamTable t) {
  Place p;
  if (!place_of(t, p)) return;
  const int i = p.i, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long blocks = (long long)(t.first[i + 1] - t.first[i] - 1) * (kAdamChunk / kAdamBlock) +
                           (t.tail[i] + kAdamBlock - 1) / kAdamBlock;
  uint32_t c[kWaveSteps];
  int top[kWaveSteps];
#pragma unroll
  for (int k = 0; k < kWaveSteps; ++k) {
    const int off = (k * (kThreads / 64) + wave) * kAdamBlock;
    c[k] = get_codes<NT>((const uint8_t *)t.m[i] + p.at + off + lane * 4, p.n - off - lane * 4);
    top[k] = off < p.n ? t.top[i][(SECOND ? blocks : 0) + (p.at + off) / kAdamBlock] : 0;
  }
#pragma unroll
  for (int k = 0; k < kWaveSteps; ++k) {
    const int off = (k * (kThreads / 64) + wave) * kAdamBlock;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = SECOND ? decode<255>(c[k] >> (8 * e), top[k] - 255)
                                              : decode<127>(c[k] >> (8 * e), top[k] - 127);
    put<NT>(t.w[i], 1, p.at + off + lane * 4, p.n - off - lane * 4, v);
  }
  end_of_stores();
}

}  // namespace

hipError_t launch_adamw(const AdamTable &t, const AdamArgs &a, bool bits8, bool stream, hipStream_t s) {
  const dim3 grid = group_grid(t.first[t.n]), threads(kThreads);
  if (bits8 && stream)
    hipLaunchKernelGGL((k_adamw<true, true>), grid, threads, 0, s, t, a);
  else if (bits8)
    hipLaunchKernelGGL((k_adamw<true, false>), grid, threads, 0, s, t, a);
  else if (stream)
    hipLaunchKernelGGL((k_adamw<false, true>), grid, threads, 0, s, t, a);
  else
    hipLaunchKernelGGL((k_adamw<false, false>), grid, threads, 0, s, t, a);
  return hipGetLastError();
}

hipError_t launch_adamw_values(const AdamTable &t, bool second, bool stream, hipStream_t s) {
  const dim3 grid = group_grid(t.first[t.n]), threads(kThreads);
  if (second && stream)
    hipLaunchKernelGGL((k_values<true, true>), grid, threads, 0, s, t);
  else if (second)
    hipLaunchKernelGGL((k_values<true, false>), grid, threads, 0, s, t);
  else if (stream)
    hipLaunchKernelGGL((k_values<false, true>), grid, threads, 0, s, t);
  else
    hipLaunchKernelGGL((k_values<false, false>), grid, threads, 0, s, t);
  return hipGetLastError();
}

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
#include "grid.h"

namespace {

constexpr int kThreads = 256, kWaveSteps = kAdamChunk / kAdamBlock / (kThreads / 64);

// n of 4 elements as fp32, the rest zero
__device__ __forceinline__ void get4(const float *p, int n, float (&v)[4]) {
  if (n >= 4) {
    __builtin_memcpy(v, p, 16);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : 0.f;
}
__device__ __forceinline__ void get4(const bf16_t *p, int n, float (&v)[4]) {
  if (n >= 4) {
    uint32_t u[2];
    __builtin_memcpy(u, p, 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < n ? bf16_to_f32(p[i]) : 0.f;
}
__device__ __forceinline__ void put4(float *p, int n, const float (&v)[4]) {
  if (n >= 4) {
    __builtin_memcpy(p, v, 16);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) p[i] = v[i];
}
__device__ __forceinline__ void put4(bf16_t *p, int n, const float (&v)[4]) {
  if (n >= 4) {
    const uint32_t u[2] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    __builtin_memcpy(p, u, 8);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) p[i] = f32_to_bf16(v[i]);
}
// four codes, the first in the low byte
__device__ __forceinline__ uint32_t get_codes(const uint8_t *p, int n) {
  uint32_t u = 0;
  if (n >= 4) {
    __builtin_memcpy(&u, p, 4);
    return u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) u |= (uint32_t)p[i] << (8 * i);
  return u;
}
__device__ __forceinline__ void put_codes(uint8_t *p, int n, uint32_t u) {
  if (n >= 4) {
    __builtin_memcpy(p, &u, 4);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) p[i] = (uint8_t)(u >> (8 * i));
}

// A tensor that is fp32 or bf16 (a branch all threads take alike).
__device__ __forceinline__ void get_any(const void *p, int f32, long long at, int n, float (&v)[4]) {
  if (f32)
    get4(reinterpret_cast<const float *>(p) + at, n, v);
  else
    get4(reinterpret_cast<const bf16_t *>(p) + at, n, v);
}
__device__ __forceinline__ void put_any(void *p, int f32, long long at, int n, const float (&v)[4]) {
  if (f32)
    put4(reinterpret_cast<float *>(p) + at, n, v);
  else
    put4(reinterpret_cast<bf16_t *>(p) + at, n, v);
}

// 32 bits of the element numbers: two rounds of multiplication by an odd
// constant and a shift, which reach every bit of the result.
__device__ __forceinline__ uint32_t mix(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x6C8E9CF5u;
  h = (h ^ (h >> 13)) * 0x51ED2701u;
  return h ^ (h >> 16);
}
constexpr uint32_t kGolden = 0x9E3779B1u;  // 2^32 by the golden ratio, odd

template <int MOST>
__device__ __forceinline__ float decode(uint32_t c, int top) {
  const int k = top - MOST + (int)(c & MOST);
  const uint32_t u = (c & MOST) && k > 0 ? (uint32_t)k << 20 : 0u;
  return __uint_as_float(MOST == 127 ? u | (c & 128u) << 24 : u);
}

constexpr uint32_t kQuietNan = 0x7FC00000u;  // every NaN's pattern here, so that tops stay below 2^11

__device__ __forceinline__ uint32_t magnitude(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < kQuietNan ? u : kQuietNan;
}

// The code of x under top T with 16 random bits r.
template <int MOST>
__device__ __forceinline__ uint32_t encode(float x, int top, uint32_t r) {
  const uint32_t mag = magnitude(x);
  int c = (int)((mag + (r << 4)) >> 20) - top + MOST;
  if (c < 1) {  // below the block's smallest value
    if (MOST == 127) {
      const int k = top - MOST + 1;
      const float least = __uint_as_float(k > 0 ? (uint32_t)k << 20 : 0u);
      c = __uint_as_float(mag) >= ((float)r + 0.5f) * 0x1p-16f * least;
    } else {
      c = 1;
    }
  }
  if (mag == 0) c = 0;
  return MOST == 127 && c > 0 && x < 0.f ? (uint32_t)c | 128u : (uint32_t)c;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t w = (uint32_t)__shfl_xor((int)v, o);
    v = v > w ? v : w;
  }
  return v;
}

// What all elements of a step share.
struct Step {
  double factor;           // of the gradients
  float lr1, root2, eps;   // lr / (1 - b1^t), (1 - b2^t)^-1/2
  float shrink;            // lr decay
  uint32_t key;
  bool clipped;
};

__device__ __forceinline__ Step step_of(const AdamArgs &a) {
  Step s;
  const long long t = a.step_dev ? *a.step_dev : a.step;
  const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
  // 1 - b^t without its cancellation
  const double c1 = -expm1((double)t * a.log1), c2 = -expm1((double)t * a.log2);
  s.lr1 = (float)(lr / c1);
  s.root2 = (float)(1.0 / sqrt(c2));
  s.eps = (float)a.eps;
  s.shrink = (float)(lr * a.decay);
  s.key = mix(a.seed + kGolden * mix((uint32_t)t));
  s.factor = 1.0;
  s.clipped = false;
  if (a.norm) {
    const double n = (double)*a.norm;
    s.clipped = n > a.tau && n <= 3.4028234663852886e38;  // a norm that is not finite clips nothing
    if (s.clipped) s.factor = a.tau / n;
  }
  return s;
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

template <bool BITS8>
__global__ __launch_bounds__(kThreads) void k_adamw(AdamTable t, AdamArgs a) {
  Place p;
  if (!place_of(t, p)) return;
  const Step s = step_of(a);
  const int i = p.i, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int w_f32 = t.w_f32[i], g_f32 = t.g_f32[i];
  const double b1 = a.beta1, b2 = a.beta2;
  const float b1f = (float)b1, b2f = (float)b2, o1 = (float)(1.0 - b1), o2 = (float)(1.0 - b2);
  const uint32_t key = BITS8 ? mix(s.key + kGolden * (uint32_t)(t.tensor0 + i + 1)) : 0u;
  long long blocks = 0;
  if (BITS8) blocks = (long long)(t.first[i + 1] - t.first[i] - 1) * (kAdamChunk / kAdamBlock) +
                      (t.tail[i] + kAdamBlock - 1) / kAdamBlock;
#pragma unroll 2
  for (int k = 0; k < kWaveSteps; ++k) {
    const int off = (k * (kThreads / 64) + wave) * kAdamBlock;  // the wave's block of this step
    if (off >= p.n) break;
    const long long at = p.at + off + lane * 4;
    const int left = p.n - off - lane * 4;
    float w[4], g[4], m[4], v[4];
    get_any(t.w[i], w_f32, at, left, w);
    get_any(t.g[i], g_f32, at, left, g);
    const long long block = (p.at + off) / kAdamBlock;
    if (BITS8) {
      const uint32_t cm = get_codes((const uint8_t *)t.m[i] + at, left), cv = get_codes((const uint8_t *)t.v[i] + at, left);
      const int tm = t.top[i][block], tv = t.top[i][blocks + block];
      uint32_t mm = 0, mv = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const double x = s.clipped ? (double)g[e] * s.factor : (double)g[e];
        m[e] = (float)(b1 * (double)decode<127>(cm >> (8 * e), tm) + (1.0 - b1) * x);
        v[e] = (float)(b2 * (double)decode<255>(cv >> (8 * e) & 255u, tv) + (1.0 - b2) * x * x);
        mm = max(mm, magnitude(m[e]));
        mv = max(mv, magnitude(v[e]));
      }
      const int um = (int)((wave_max(mm) + 0xFFFFFu) >> 20), uv = (int)((wave_max(mv) + 0xFFFFFu) >> 20);
      if (lane == 0) {
        t.top[i][block] = (int16_t)um;
        t.top[i][blocks + block] = (int16_t)uv;
      }
      uint32_t nm = 0, nv = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t r = mix(key + (uint32_t)(at + e) * kGolden);
        nm |= encode<127>(m[e], um, r & 0xFFFFu) << (8 * e);
        nv |= encode<255>(v[e], uv, r >> 16) << (8 * e);
      }
      put_codes((uint8_t *)t.m[i] + at, left, nm);
      put_codes((uint8_t *)t.v[i] + at, left, nv);
    } else {
      get4((const float *)t.m[i] + at, left, m);
      get4((const float *)t.v[i] + at, left, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = s.clipped ? (float)((double)g[e] * s.factor) : g[e];
        m[e] = fmaf(b1f, m[e], o1 * x);
        v[e] = fmaf(b2f, v[e], o2 * x * x);
      }
      put4((float *)t.m[i] + at, left, m);
      put4((float *)t.v[i] + at, left, v);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float q = s.lr1 * m[e] / (sqrtf(v[e]) * s.root2 + s.eps);
      w[e] = fmaf(-s.shrink, w[e], w[e]) - q;
    }
    put_any(t.w[i], w_f32, at, left, w);
    if (t.copy[i]) put4(t.copy[i] + at, left, w);
  }
}

template <bool SECOND>
__global__ __launch_bounds__(kThreads) void k_values(AdamTable t) {
  Place p;
  if (!place_of(t, p)) return;
  const int i = p.i, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long blocks = (long long)(t.first[i + 1] - t.first[i] - 1) * (kAdamChunk / kAdamBlock) +
                           (t.tail[i] + kAdamBlock - 1) / kAdamBlock;
#pragma unroll
  for (int k = 0; k < kWaveSteps; ++k) {
    const int off = (k * (kThreads / 64) + wave) * kAdamBlock;
    if (off >= p.n) break;
    const long long at = p.at + off + lane * 4;
    const int left = p.n - off - lane * 4;
    const uint32_t c = get_codes((const uint8_t *)t.m[i] + at, left);
    const int top = t.top[i][(SECOND ? blocks : 0) + (p.at + off) / kAdamBlock];
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = SECOND ? decode<255>(c >> (8 * e) & 255u, top) : decode<127>(c >> (8 * e) & 255u, top);
    put4((float *)t.w[i] + at, left, v);
  }
}

}  // namespace

hipError_t launch_adamw(const AdamTable &t, const AdamArgs &a, bool bits8, hipStream_t s) {
  const dim3 grid = group_grid(t.first[t.n]);
  if (bits8)
    hipLaunchKernelGGL(k_adamw<true>, grid, dim3(kThreads), 0, s, t, a);
  else
    hipLaunchKernelGGL(k_adamw<false>, grid, dim3(kThreads), 0, s, t, a);
  return hipGetLastError();
}

hipError_t launch_adamw_values(const AdamTable &t, bool second, hipStream_t s) {
  const dim3 grid = group_grid(t.first[t.n]);
  if (second)
    hipLaunchKernelGGL(k_values<true>, grid, dim3(kThreads), 0, s, t);
  else
    hipLaunchKernelGGL(k_values<false>, grid, dim3(kThreads), 0, s, t);
  return hipGetLastError();
}

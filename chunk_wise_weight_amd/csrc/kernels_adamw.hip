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
// before they become codes. fp32 sums would do for the moments, but where they
// are computed elsewhere (a replica, a resumed run on other software) another
// order of their roundings would change the last bit of every second value, and
// one bit in 2^20 is a border between two codes: some 10^-6 of the codes would
// differ at every step. In fp64 another order of the products and sums, which the
// definition leaves open, reaches the fp32 value in some 10^-8 of all cases and a
// code in some 10^-14. On this library the codes are the same on every run.
#include <type_traits>

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
// Eight elements likewise.
struct Eight {
  uint32_t u[8];
};
template <bool NT>
__device__ __forceinline__ Eight get8(const void *p, int f32, long long at, int n) {
  Eight r = {};
  if (n >= 8) {
    if (f32) {
      const float *q = reinterpret_cast<const float *>(p) + at;
      const u32x4_el a = fetch<NT, u32x4_el>(q), b = fetch<NT, u32x4_el>(q + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r.u[i] = a[i];
        r.u[4 + i] = b[i];
      }
    } else {
      const u32x4_any v = fetch<NT, u32x4_any>(reinterpret_cast<const bf16_t *>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.u[i] = v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      if (i >= n) continue;
      if (f32)
        r.u[i] = reinterpret_cast<const uint32_t *>(p)[at + i];
      else
        r.u[i / 2] |= (uint32_t)reinterpret_cast<const bf16_t *>(p)[at + i] << (16 * (i & 1));
    }
  }
  return r;
}
__device__ __forceinline__ void expand(const Eight &r, int f32, float (&v)[8]) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.u[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.u[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.u[i] & 0xffff0000u);
    }
  }
}
template <bool NT>
__device__ __forceinline__ void put8(void *p, int f32, long long at, int n, const float (&v)[8]) {
  if (n >= 8) {
    if (f32) {
      float *q = reinterpret_cast<float *>(p) + at;
      keep<NT>(q, u32x4_el{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
      keep<NT>(q + 4, u32x4_el{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
    } else {
      keep<NT>(reinterpret_cast<bf16_t *>(p) + at, u32x4_any{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                             pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])});
    }
    end_of_stores();
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      if (i >= n) continue;
      if (f32)
        reinterpret_cast<float *>(p)[at + i] = v[i];
      else
        reinterpret_cast<bf16_t *>(p)[at + i] = f32_to_bf16(v[i]);
    }
  }
}
typedef uint32_t u32x2_code __attribute__((ext_vector_type(2), aligned(1)));
struct Codes8 {
  uint32_t u[2];
};
template <bool NT>
__device__ __forceinline__ Codes8 get_codes8(const uint8_t *p, int n) {
  if (n >= 8) {
    const u32x2_code v = fetch<NT, u32x2_code>(p);
    return {{v[0], v[1]}};
  }
  Codes8 r = {};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) r.u[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
  return r;
}
template <bool NT>
__device__ __forceinline__ void put_codes8(uint8_t *p, int n, const Codes8 &c) {
  if (n >= 8) {
    keep<NT>(p, u32x2_code{c.u[0], c.u[1]});
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) p[i] = (uint8_t)(c.u[i / 4] >> (8 * (i & 3)));
}

// The value of byte e of c under a block's top, lowest = top - most. HIGH: every code but 0 stands for a pattern above 0.
template <int MOST, bool HIGH>
__device__ __forceinline__ float decode(uint32_t c, int e, int lowest) {
  const uint32_t code = c >> (8 * e) & MOST;
  const int k = lowest + (int)code;
  const uint32_t u = code ? (uint32_t)(HIGH ? k : max(k, 0)) << 20 : 0u;
  return __uint_as_float(MOST == 127 ? u | (c << (24 - 8 * e) & 0x80000000u) : u);
}

constexpr uint32_t kQuietNan = 0x7FC00000u;  // every NaN's pattern here, so that tops stay below 2^11

// The code of x, of magnitude mag, under a block's lowest = top - most, with 16 random bits r. HIGH: as above, and no
// NaN among the block's.
template <int MOST, bool HIGH>
__device__ __forceinline__ uint32_t encode(float x, uint32_t mag, int lowest, uint32_t r) {
  if (!HIGH) mag = min(mag, kQuietNan);
  int c = (int)((mag + (r << 4)) >> 20) - lowest;
  if (MOST == 255) return (uint32_t)(HIGH ? max(c, (int)min(mag, 1u)) : mag ? max(c, 1) : 0);
  uint32_t sign = __float_as_uint(x) >> 24 & 128u;
  if (!HIGH || __any(c < 1)) {  // below the block's smallest value, which few are
    const float least = __uint_as_float(lowest > -1 ? (uint32_t)(lowest + 1) << 20 : 0u);
    const int low = __uint_as_float(mag) >= ((float)r + 0.5f) * 0x1p-16f * least;
    c = mag == 0 ? 0 : c < 1 ? low : c;
    sign = c ? sign : 0;
  }
  return (uint32_t)c | sign;
}

// The largest of the values of a wave's lower or upper 32 lanes, in each of them: by rotations within the rows of 16
// lanes, then between two rows.
__device__ __forceinline__ uint32_t half_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, true));  // row_ror:8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, true));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max((uint32_t)a[0], (uint32_t)a[1]);
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

// sqrt(v) by the hardware's root (1 ulp), with SMALL also of the denormals, which it may take as 0: their roots times
// root2 are below 2^-63 root2, half a step of an eps from 2 10^-12 root2 on.
template <bool SMALL>
__device__ __forceinline__ float root(float v) {
  if (!SMALL) return __builtin_amdgcn_sqrtf(v);
  const bool tiny = v < 0x1p-96f;
  return __builtin_amdgcn_sqrtf(tiny ? v * 0x1p64f : v) * (tiny ? 0x1p-32f : 1.f);
}
__device__ __forceinline__ bool small_eps(float eps, float root2) { return eps < 2e-12f * root2; }

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

// The betas and the gradients' factor.
struct Rates {
  double b1, b2, factor;
  bool clipped;
};
__device__ __forceinline__ Rates rates_of(const AdamArgs &a) {
  Rates r{a.beta1, a.beta2, 1.0, false};
  if (a.norm) {
    const double n = (double)*a.norm;
    r.clipped = n > a.tau && n <= 3.4028234663852886e38;  // a norm that is not finite clips nothing
    if (r.clipped) r.factor = a.tau / n;
  }
  return r;
}
// With SMALL the denominator may be a denormal, which the hardware's reciprocal may take as 0 (and 0 / eps would be 0
// times infinity); below 2^-96 it is scaled, and the moment alike before lr1 makes it smaller.
template <bool SMALL>
__device__ __forceinline__ float moved(float w, float m, float v, const AdamStep &s, float eps) {
  const float d = fmaf(root<SMALL>(v), s.root2, eps);
  float q = s.lr1 * m * __builtin_amdgcn_rcpf(d);
  if (SMALL && d < 0x1p-96f) q = s.lr1 * (m * 0x1p96f * __builtin_amdgcn_rcpf(d * 0x1p96f));
  return fmaf(-s.shrink, w, w) - q;
}
// f(std::true_type) where eps is small, else f(std::false_type): all threads take one branch, and it is the elements' loop
// that is in it (a branch for each of them costs the 8-bit form 3 %).
template <class F>
__device__ __forceinline__ void by_eps(float eps, float root2, F &&f) {
  if (small_eps(eps, root2))
    f(std::true_type{});
  else
    f(std::false_type{});
}

// beta x, rounded once; an infinity's small part must not meet its large one as another infinity, or as 0 times it
__device__ __forceinline__ float decayed(const AdamDecay &b, float x) {
  constexpr float kMost = 3.4028234663852886e38f;
  return fmaf(b.hi, x, b.lo * __builtin_amdgcn_fmed3f(x, -kMost, kMost));
}

// fp32 moments: a wave takes four blocks of a chunk, a lane four elements of each. Everything is loaded before anything
// is stored. FULL: every element of the chunk is there.
template <bool NT, bool FULL>
__device__ __forceinline__ void step_chunk(const AdamTable &t, const AdamArgs &a, const Place &p) {
  const int i = p.i, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int w_f32 = t.w_f32[i], g_f32 = t.g_f32[i];
  const long long at0 = p.at + wave * kAdamBlock + lane * 4;
  const int left0 = p.n - wave * kAdamBlock - lane * 4;
  constexpr int SKIP = kThreads / 64 * kAdamBlock;  // from a wave's block to its next
  Four w[kWaveSteps], g[kWaveSteps], m[kWaveSteps], v[kWaveSteps];
#pragma unroll
  for (int k = 0; k < kWaveSteps; ++k) {
    const long long at = at0 + k * SKIP;
    const int left = FULL ? 4 : left0 - k * SKIP;
    w[k] = get<NT>(t.w[i], w_f32, at, left);
    g[k] = get<NT>(t.g[i], g_f32, at, left);
    m[k] = get<NT>(t.m[i], 1, at, left);
    v[k] = get<NT>(t.v[i], 1, at, left);
  }
  const AdamStep s = step_of(a);
  const Rates r = rates_of(a);
  const AdamDecay b1 = a.decay1, b2 = a.decay2;
#pragma unroll
  for (int k = 0; k < kWaveSteps; ++k) {
    const long long at = at0 + k * SKIP;
    const int left = FULL ? 4 : left0 - k * SKIP;
    float x[4], mk[4], vk[4], wk[4];
    expand(g[k], g_f32, x);
    expand(w[k], w_f32, wk);
    expand(m[k], 1, mk);
    expand(v[k], 1, vk);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // the factor to the gradient first: its square may leave fp32
      const float d = r.clipped ? (float)((double)x[e] * r.factor) : x[e];
      mk[e] = fmaf(b1.rest, d, decayed(b1, mk[e]));
      vk[e] = fmaf(b2.rest * d, d, decayed(b2, vk[e]));
    }
    by_eps(a.eps, s.root2, [&](auto small) {
#pragma unroll
      for (int e = 0; e < 4; ++e) wk[e] = moved<decltype(small)::value>(wk[e], mk[e], vk[e], s, a.eps);
    });
    put<NT>(t.m[i], 1, at, left, mk);
    put<NT>(t.v[i], 1, at, left, vk);
    put<NT>(t.w[i], w_f32, at, left, wk);
    if (t.copy[i]) put<NT>(t.copy[i], 0, at, left, wk);
  }
  end_of_stores();
}

// 8-bit moments: half a wave takes a block, a lane eight elements of it, two blocks one after the other. (277M bf16
// weights: 660 us. When this form took 680, four elements per lane took 729 and a block each for 512 threads 750. 66 vector
// instructions per element are 480 us of it, the bytes at the rate of the fp32 form 490.)
constexpr int kHalfSteps = kAdamChunk / kAdamBlock / (kThreads / 32);

template <bool NT, bool FULL>
__device__ __forceinline__ void step_chunk8(const AdamTable &t, const AdamArgs &a, const Place &p) {
  const int i = p.i, lane = threadIdx.x & 31, half = threadIdx.x >> 5;
  const int w_f32 = t.w_f32[i], g_f32 = t.g_f32[i];
  constexpr int SKIP = kThreads / 32 * kAdamBlock;  // from a half's block to its next
  const long long at0 = p.at + half * kAdamBlock + lane * 8;
  const int left0 = p.n - half * kAdamBlock - lane * 8;
  const long long block0 = p.at / kAdamBlock + half;
  const long long blocks = (long long)(t.first[i + 1] - t.first[i] - 1) * (kAdamChunk / kAdamBlock) +
                           (t.tail[i] + kAdamBlock - 1) / kAdamBlock;
  Eight w[kHalfSteps], g[kHalfSteps];
  Codes8 m[kHalfSteps], v[kHalfSteps];
  int tm[kHalfSteps], tv[kHalfSteps];
#pragma unroll
  for (int k = 0; k < kHalfSteps; ++k) {
    const long long at = at0 + k * SKIP;
    const int left = FULL ? 8 : left0 - k * SKIP;
    w[k] = get8<NT>(t.w[i], w_f32, at, left);
    g[k] = get8<NT>(t.g[i], g_f32, at, left);
    m[k] = get_codes8<NT>((const uint8_t *)t.m[i] + at, left);
    v[k] = get_codes8<NT>((const uint8_t *)t.v[i] + at, left);
    const bool there = FULL || left + lane * 8 > 0;  // the block is there
    const long long block = block0 + k * (kThreads / 32);
    tm[k] = there ? t.top[i][block] : 0;
    tv[k] = there ? t.top[i][blocks + block] : 0;
  }
  const AdamStep s = step_of(a);
  const Rates r = rates_of(a);
  // fp64 holds the factor's square with the betas
  const double b1 = r.b1, b2 = r.b2, o1 = (1.0 - b1) * r.factor, o2 = (1.0 - b2) * r.factor * r.factor;
  const uint32_t key = adam_mix(s.key + kGolden * (uint32_t)(t.tensor0 + i + 1));
#pragma unroll
  for (int k = 0; k < kHalfSteps; ++k) {
    const long long at = at0 + k * SKIP;
    const int left = FULL ? 8 : left0 - k * SKIP;
    const bool there = FULL || left + lane * 8 > 0;
    float x[8], mk[8], vk[8], wk[8];
    expand(g[k], g_f32, x);
    // both blocks' tops far above the smallest fp32 number, as they are but for moments below 10^-28 or of 0
    const bool high = !__any(tm[k] < 128 || tv[k] < 256);
    auto recur = [&](auto hi) {
      constexpr bool HIGH = decltype(hi)::value;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double d = (double)x[e];
        mk[e] = (float)(b1 * (double)decode<127, HIGH>(m[k].u[e / 4], e % 4, tm[k] - 127) + o1 * d);
        vk[e] = (float)(b2 * (double)decode<255, HIGH>(v[k].u[e / 4], e % 4, tv[k] - 255) + o2 * d * d);
      }
    };
    if (high)
      recur(std::true_type{});
    else
      recur(std::false_type{});
    uint32_t mm = 0, mv = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mm = max(mm, __float_as_uint(mk[e]) & 0x7fffffffu);
      mv = max(mv, __float_as_uint(vk[e]) & 0x7fffffffu);
    }
    mm = half_max(mm);
    mv = half_max(mv);
    const int um = (int)((min(mm, kQuietNan) + 0xFFFFFu) >> 20), uv = (int)((min(mv, kQuietNan) + 0xFFFFFu) >> 20);
    if (lane == 0 && there) {
      const long long block = block0 + k * (kThreads / 32);
      t.top[i][block] = (int16_t)um;
      t.top[i][blocks + block] = (int16_t)uv;
    }
    Codes8 nm, nv;
    const uint32_t place = key + (uint32_t)at * kGolden;
    auto codes = [&](auto hi) {
      constexpr bool HIGH = decltype(hi)::value;
      nm = nv = Codes8{};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t rnd = adam_mix(place + e * kGolden);
        nm.u[e / 4] |= encode<127, HIGH>(mk[e], __float_as_uint(mk[e]) & 0x7fffffffu, um - 127, rnd & 0xFFFFu) << (8 * (e % 4));
        nv.u[e / 4] |= encode<255, HIGH>(vk[e], __float_as_uint(vk[e]) & 0x7fffffffu, uv - 255, rnd >> 16) << (8 * (e % 4));
      }
    };
    if (!__any(um < 128 || uv < 256 || mm > 0x7f800000u || mv > 0x7f800000u))
      codes(std::true_type{});
    else
      codes(std::false_type{});
    put_codes8<NT>((uint8_t *)t.m[i] + at, left, nm);
    put_codes8<NT>((uint8_t *)t.v[i] + at, left, nv);
    expand(w[k], w_f32, wk);
    by_eps(a.eps, s.root2, [&](auto small) {
#pragma unroll
      for (int e = 0; e < 8; ++e) wk[e] = moved<decltype(small)::value>(wk[e], mk[e], vk[e], s, a.eps);
    });
    put8<NT>(t.w[i], w_f32, at, left, wk);
    if (t.copy[i]) put8<NT>(t.copy[i], 0, at, left, wk);
  }
  end_of_stores();
}

template <bool BITS8, bool NT>
__global__ __launch_bounds__(kThreads) void k_adamw(AdamTable t, AdamArgs a) {
  Place p;
  if (!place_of(t, p)) return;
  if (p.n == kAdamChunk) {
    if constexpr (BITS8)
      step_chunk8<NT, true>(t, a, p);
    else
      step_chunk<NT, true>(t, a, p);
  } else {
    if constexpr (BITS8)
      step_chunk8<NT, false>(t, a, p);
    else
      step_chunk<NT, false>(t, a, p);
  }
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
    for (int e = 0; e < 4; ++e) v[e] = SECOND ? decode<255, false>(c[k], e, top[k] - 255) : decode<127, false>(c[k], e, top[k] - 127);
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

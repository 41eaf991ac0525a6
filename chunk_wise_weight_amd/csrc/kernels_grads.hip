// The 2-norm of many tensors together, N = (sum of g^2)^1/2, and their scaling
// by min(1, tau / N).
//
// Squares are formed and added in fp64: fp32 squares leave its range for
// |g| > 1e19 or < 1e-19 (clipped updates of the layer are 1e-9 and less), and
// the sums run over up to billions of terms. The conversions cost vector
// instructions, not time: the kernels are bound by reading the gradients. Each
// workgroup adds its chunks in a fixed order, and one workgroup adds the
// workgroups' sums in a fixed order, so a call's bits do not change.
#include "grads.h"
#include "grid.h"

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ double wave_sum(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// 16 bytes as they lie in memory, at any element: four fp32 or eight bf16.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <bool NT>
__device__ __forceinline__ u32x4_any load16(const void *p) {
  const u32x4_any *q = reinterpret_cast<const u32x4_any *>(p);
  return NT ? __builtin_nontemporal_load(q) : *q;
}
template <bool NT>
__device__ __forceinline__ void store16(void *p, u32x4_any v) {
  u32x4_any *q = reinterpret_cast<u32x4_any *>(p);
  if (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

__device__ __forceinline__ double square(float v) { return (double)v * (double)v; }
__device__ __forceinline__ float lower(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float upper(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_to_f32(v); }

template <typename T>
__device__ __forceinline__ double squares16(u32x4_any v) {
  double s = 0.0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    s += sizeof(T) == 4 ? square(__uint_as_float(v[j])) : square(lower(v[j])) + square(upper(v[j]));
  return s;
}
// v tau / N with the factor as mantissa and exponent: as one fp32 number it
// would lose its bits below 1e-38, where tau is small and N large.
__device__ __forceinline__ float scaled(float v, GradFactor f) { return ldexpf(v * f.mantissa, f.exponent); }

template <typename T>
__device__ __forceinline__ u32x4_any scaled16(u32x4_any v, GradFactor f) {
  u32x4_any r;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r[j] = sizeof(T) == 4 ? __float_as_uint(scaled(__uint_as_float(v[j]), f))
                          : pack_bf16x2(scaled(lower(v[j]), f), scaled(upper(v[j]), f));
  return r;
}

// 16-byte pieces of a full chunk per thread, and elements of a chunk
constexpr int kPieces = kGradBytes / 16 / kThreads;
template <typename T>
constexpr int kChunk = kGradBytes / sizeof(T);

// the sum of squares of up to a chunk
template <typename T, bool NT>
__device__ __forceinline__ double chunk_squares(const T *p, int n) {
  constexpr int E = 16 / sizeof(T), P = kPieces;
  double s = 0.0;
  if (n == kChunk<T>) {
    u32x4_any v[P];
#pragma unroll
    for (int k = 0; k < P; ++k) v[k] = load16<NT>(p + (k * kThreads + threadIdx.x) * E);
#pragma unroll
    for (int k = 0; k < P; ++k) s += squares16<T>(v[k]);
    return s;
  }
  for (int i = threadIdx.x * E; i + E <= n; i += kThreads * E) s += squares16<T>(load16<NT>(p + i));
  if ((int)threadIdx.x < n % E) s += square(to_f32(p[n / E * E + threadIdx.x]));
  return s;
}

__device__ __forceinline__ void put1(float *q, float v) { *q = v; }
__device__ __forceinline__ void put1(bf16_t *q, float v) { *q = f32_to_bf16(v); }

template <bool NT>
constexpr int kScaleParts = NT ? 4 : 1;

// one of PARTS parts of up to a chunk, scaled
template <typename T, bool NT, int PARTS>
__device__ __forceinline__ void chunk_scale(const T *p, T *q, int n, int part, GradFactor f) {
  constexpr int E = 16 / sizeof(T), N = kChunk<T> / PARTS;  // elements of a part
  const int lo = part * N, hi = lo + N < n ? lo + N : n;
  if (hi - lo == N) {
    u32x4_any v[kPieces / PARTS];
#pragma unroll
    for (int k = 0; k < kPieces / PARTS; ++k) v[k] = load16<NT>(p + lo + (k * kThreads + threadIdx.x) * E);
#pragma unroll
    for (int k = 0; k < kPieces / PARTS; ++k)
      store16<NT>(q + lo + (k * kThreads + threadIdx.x) * E, scaled16<T>(v[k], f));
    return;
  }
  for (int i = lo + threadIdx.x * E; i + E <= hi; i += kThreads * E)
    store16<NT>(q + i, scaled16<T>(load16<NT>(p + i), f));
  if (hi <= lo) return;  // a part past the tensor's end
  const int rest = hi - (hi - lo) % E + threadIdx.x;
  if (rest < hi) put1(q + rest, scaled(to_f32(p[rest]), f));
}

// part[blockIdx.x]: the sum of squares of chunks blockIdx.x, + gridDim.x, ...
// 539M fp32 values (2.16 GB) take 315 us, 6.9 TB/s, which is what reading alone
// reaches here (425 us in chunks of 128 KiB and through the caches).
template <bool NT>
__global__ __launch_bounds__(kThreads) void k_squares(GradTable t, double *part) {
  __shared__ double red[kThreads / 64];
  double s = 0.0;
  int i = 0;  // the chunk's tensor: chunks only go up
  for (uint32_t c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    while (c >= t.first[i + 1]) ++i;
    const bool last = c + 1 == t.first[i + 1];
    const long long at = (long long)(c - t.first[i]) * kGradBytes;
    if (t.f32[i])
      s += chunk_squares<float, NT>(reinterpret_cast<const float *>((const char *)t.g[i] + at),
                                    last ? (int)t.tail[i] : kChunk<float>);
    else
      s += chunk_squares<bf16_t, NT>(reinterpret_cast<const bf16_t *>((const char *)t.g[i] + at),
                                     last ? (int)t.tail[i] : kChunk<bf16_t>);
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kThreads / 64; ++w) s += red[w];
  part[blockIdx.x] = s;
}

// The norm from the workgroups' sums, and the factor min(1, tau / norm): 1
// where the norm is not finite (a factor below 1 has a mantissa below 1 or a
// negative exponent).
__global__ __launch_bounds__(1024) void k_norm(const double *part, int n, float tau, float *norm, GradFactor *factor) {
  __shared__ double red[16];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) s += part[i];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 16; ++w) s += red[w];
  const double v = sqrt(s);
  *norm = (float)v;
  if (!factor) return;
  GradFactor f{1.f, 0};
  if (v > (double)tau && v <= 1.7e308) {
    const double m = frexp((double)tau / v, &f.exponent);
    f.mantissa = (float)m;
  }
  *factor = f;
}

// A workgroup per chunk, or, of gradients past the caches (NT), per page of 4
// KiB, which workgroups on different dies should not share: 539M fp32 values
// (4.3 GB) take 650 us, 6.6 TB/s, as a copy does; 715 by chunks, 850 with
// workgroups that stay and stride over the chunks (a wave's loads would wait
// behind its own stores), 760 through the caches. Taking the chunks in the
// opposite order, to find the last ones read still cached, gains nothing at
// any size. Where most calls clip nothing and only look, smaller steps cost:
// 70M bf16 values in place take 33 us by chunks and 38 by pages.
template <bool NT>
__global__ __launch_bounds__(kThreads) void k_scale(GradTable t, const GradFactor *factor) {
  constexpr int PARTS = kScaleParts<NT>;
  const long long g = group_index();
  if (g >= (long long)t.first[t.n] * PARTS) return;
  const uint32_t c = (uint32_t)(g / PARTS);
  const int part = (int)(g % PARTS);
  int lo = 0, hi = t.n - 1;  // the tensor of the chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  const GradFactor f = *factor;
  if (f.mantissa == 1.f && f.exponent == 0 && t.out[lo] == t.g[lo]) return;  // in place, and not clipped
  const bool last = c + 1 == t.first[lo + 1];
  const long long at = (long long)(c - t.first[lo]) * kGradBytes;
  const char *p = (const char *)t.g[lo] + at;
  char *q = (char *)t.out[lo] + at;
  if (t.f32[lo])
    chunk_scale<float, NT, PARTS>(reinterpret_cast<const float *>(p), reinterpret_cast<float *>(q),
                           last ? (int)t.tail[lo] : kChunk<float>, part, f);
  else
    chunk_scale<bf16_t, NT, PARTS>(reinterpret_cast<const bf16_t *>(p), reinterpret_cast<bf16_t *>(q),
                            last ? (int)t.tail[lo] : kChunk<bf16_t>, part, f);
}

}  // namespace

hipError_t launch_grad_squares(const GradTable &t, double *part, int groups, bool stream, hipStream_t s) {
  if (stream)
    hipLaunchKernelGGL(k_squares<true>, dim3(groups), dim3(kThreads), 0, s, t, part);
  else
    hipLaunchKernelGGL(k_squares<false>, dim3(groups), dim3(kThreads), 0, s, t, part);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const double *part, int n, float tau, float *norm, GradFactor *factor, hipStream_t s) {
  hipLaunchKernelGGL(k_norm, dim3(1), dim3(1024), 0, s, part, n, tau, norm, factor);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradTable &t, const GradFactor *factor, bool stream, hipStream_t s) {
  const dim3 grid = group_grid((long long)t.first[t.n] * (stream ? kScaleParts<true> : kScaleParts<false>));
  if (stream)
    hipLaunchKernelGGL(k_scale<true>, grid, dim3(kThreads), 0, s, t, factor);
  else
    hipLaunchKernelGGL(k_scale<false>, grid, dim3(kThreads), 0, s, t, factor);
  return hipGetLastError();
}

// The 2-norm of many tensors together, N = (sum of g^2)^1/2, and their scaling
// by min(1, tau / N).
//
// Squares are formed and added in fp64: fp32 squares leave its range for
// |g| > 1e19 or < 1e-19 (clipped updates of the layer are 1e-9 and less), and
// the sums run over up to billions of terms. The conversions cost vector
// instructions, not time: the kernels are bound by reading the gradients. Each
// workgroup adds its chunks in a fixed order, and everyone who needs the norm
// adds the workgroups' sums in a fixed order, so a call's bits do not change.
#include "grads.h"
#include "vec8.h"

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ double wave_sum(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// the sum over the workgroup, in every thread
__device__ __forceinline__ double group_sum(double v, double *red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kThreads / 64; ++w) s += red[w];
  return s;
}

// the tensor that chunk c belongs to
__device__ __forceinline__ int tensor_of(const GradTable &t, uint32_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ double squares(const T *p, uint32_t n) {
  double s = 0.0;
#pragma unroll 4
  for (uint32_t i = threadIdx.x * 8; i + 8 <= n; i += kThreads * 8) {
    float v[8];
    load_w(p + i, true, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (double)v[j] * (double)v[j];
  }
  if (threadIdx.x < n % 8) {
    float v[1];
    load_w(p + n / 8 * 8 + threadIdx.x, true, v);
    s += (double)v[0] * (double)v[0];
  }
  return s;
}

template <typename T>
__device__ __forceinline__ void scale(const T *p, T *q, uint32_t n, float c) {
#pragma unroll 4
  for (uint32_t i = threadIdx.x * 8; i + 8 <= n; i += kThreads * 8) {
    float v[8];
    load_w(p + i, true, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= c;
    store_w(q + i, true, v);
  }
  if (threadIdx.x < n % 8) {
    const uint32_t i = n / 8 * 8 + threadIdx.x;
    float v[1];
    load_w(p + i, true, v);
    v[0] *= c;
    store_w(q + i, true, v);
  }
}

__global__ __launch_bounds__(kThreads) void k_squares(GradTable t, double *part) {
  __shared__ double red[kThreads / 64];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const uint32_t n = c + 1 == t.first[i + 1] ? t.tail[i] : t.chunk;
    const long long at = (long long)(c - t.first[i]) * t.chunk;
    s += t.f32[i] ? squares(reinterpret_cast<const float *>(t.g[i]) + at, n)
                  : squares(reinterpret_cast<const bf16_t *>(t.g[i]) + at, n);
  }
  s = group_sum(s, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double total_norm(const double *part, int n, double *red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += part[i];
  return sqrt(group_sum(s, red));
}

__global__ __launch_bounds__(kThreads) void k_norm(const double *part, int n, float *norm) {
  __shared__ double red[kThreads / 64];
  const double v = total_norm(part, n, red);
  if (threadIdx.x == 0) *norm = (float)v;
}

__global__ __launch_bounds__(kThreads) void k_scale(GradTable t, const double *part, int n, float tau, float *norm) {
  __shared__ double red[kThreads / 64];
  const double v = total_norm(part, n, red);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  const bool clip = v > (double)tau && v <= 1.7e308;
  const float f = clip ? (float)((double)tau / v) : 1.f;
  for (uint32_t c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    if (!clip && t.out[i] == t.g[i]) continue;
    const uint32_t m = c + 1 == t.first[i + 1] ? t.tail[i] : t.chunk;
    const long long at = (long long)(c - t.first[i]) * t.chunk;
    if (t.f32[i])
      scale(reinterpret_cast<const float *>(t.g[i]) + at, reinterpret_cast<float *>(t.out[i]) + at, m, f);
    else
      scale(reinterpret_cast<const bf16_t *>(t.g[i]) + at, reinterpret_cast<bf16_t *>(t.out[i]) + at, m, f);
  }
}

}  // namespace

hipError_t launch_grad_squares(const GradTable &t, double *part, int groups, hipStream_t s) {
  hipLaunchKernelGGL(k_squares, dim3(groups), dim3(kThreads), 0, s, t, part);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const double *part, int n, float *norm, hipStream_t s) {
  hipLaunchKernelGGL(k_norm, dim3(1), dim3(kThreads), 0, s, part, n, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradTable &t, const double *part, int n, float tau, float *norm, int groups,
                             hipStream_t s) {
  hipLaunchKernelGGL(k_scale, dim3(groups), dim3(kThreads), 0, s, t, part, n, tau, norm);
  return hipGetLastError();
}

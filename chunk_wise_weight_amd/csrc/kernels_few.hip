// The forward products of a few rows, as when sequences decode: every weight is
// read once, and its bytes are what counts.
//
// A workgroup takes 16 rows of the weights (with a pair 16 of each matrix) and
// up to 64 tokens, its waves take turns along k. Fragments come straight from
// memory: lane l holds 16 bytes of weight row l % 16 and of token l % 16, at
// the same k, a step of 64 bytes of every row. Several steps are loaded before
// the first is multiplied, so that a wave has 8 KB of weights in flight. The
// waves' sums are added in LDS, in their order. Rows and tokens past the end
// are read as the last one's, and their sums are not stored.
#include <algorithm>

#include "linear_dev.h"

namespace {

__device__ __forceinline__ void mma(f32x4 &acc, const Raw8<bf16_t> &a, const Raw8<bf16_t> &b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4 &acc, const f32x4 &a, const f32x4 &b) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], acc, 0, 0, 0);
}

// 16 bytes of a row
template <typename T>
struct Piece;
template <>
struct Piece<bf16_t> {
  typedef Raw8<bf16_t> type;
};
template <>
struct Piece<float> {
  typedef f32x4 type;
};
template <typename T>
__device__ __forceinline__ typename Piece<T>::type piece(const T *p) {
  typename Piece<T>::type v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
// n of its elements, the rest zero
template <typename T>
__device__ __forceinline__ typename Piece<T>::type piece(const T *p, int n) {
  T e[16 / sizeof(T)] = {};
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(T); ++i)
    if (i < n) e[i] = p[i];
  typename Piece<T>::type v;
  __builtin_memcpy(&v, e, 16);
  return v;
}

template <typename T, typename O, bool PAIR, int FJ>
__global__ __launch_bounds__(1024) void k_few(GemmArgs g) {
  extern __shared__ __attribute__((aligned(16))) f32x4 sums[];  // [fragment][wave][lane]
  constexpr int E = 16 / sizeof(T), STEP = 4 * E, FI = PAIR ? 2 : 1, U = FJ == 1 ? 8 : 4;
  typedef typename Piece<T>::type P;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const long long i0 = (long long)blockIdx.x * 16;
  const long long row = i0 + (lane & 15) < g.ni ? i0 + (lane & 15) : g.ni - 1;
  const int nk = (int)g.nk, kl = (lane >> 4) * E;
  const T *a[FI], *b[FJ];
#pragma unroll
  for (int x = 0; x < FI; ++x) a[x] = reinterpret_cast<const T *>(g.a[x]) + row * g.lda + kl;
#pragma unroll
  for (int y = 0; y < FJ; ++y) {
    const long long j = y * 16 + (lane & 15);
    b[y] = reinterpret_cast<const T *>(g.b[0]) + (j < g.nj ? j : g.nj - 1) * g.ldb + kl;
  }
  f32x4 acc[FI][FJ];
#pragma unroll
  for (int x = 0; x < FI; ++x)
#pragma unroll
    for (int y = 0; y < FJ; ++y) acc[x][y] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int full = nk / STEP;  // whole steps
  int s = w * U;
  for (; s + U <= full; s += nw * U) {
    P fa[U][FI], fb[U][FJ];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int x = 0; x < FI; ++x) fa[u][x] = piece(a[x] + (s + u) * STEP);
#pragma unroll
      for (int y = 0; y < FJ; ++y) fb[u][y] = piece(b[y] + (s + u) * STEP);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) mma(acc[x][y], fa[u][x], fb[u][y]);
  }
  // the run of less than U steps, and what is left of k behind them: the wave's whose turn it is
  if (s < full || (s == full && nk % STEP)) {
    for (; s < full; ++s)
#pragma unroll
      for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) mma(acc[x][y], piece(a[x] + s * STEP), piece(b[y] + s * STEP));
    const int n = nk - full * STEP - kl;  // of this lane's piece
    if (nk % STEP) {
      P fa[FI], fb[FJ];
#pragma unroll
      for (int x = 0; x < FI; ++x) fa[x] = piece(a[x] + full * STEP, n);
#pragma unroll
      for (int y = 0; y < FJ; ++y) fb[y] = piece(b[y] + full * STEP, n);
#pragma unroll
      for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) mma(acc[x][y], fa[x], fb[y]);
    }
  }
#pragma unroll
  for (int x = 0; x < FI; ++x)
#pragma unroll
    for (int y = 0; y < FJ; ++y) sums[((x * FJ + y) * nw + w) * 64 + lane] = acc[x][y];
  __syncthreads();
  for (int y = w; y < FJ; y += nw) {
    f32x4 t[FI];
#pragma unroll
    for (int x = 0; x < FI; ++x) {
      t[x] = sums[(x * FJ + y) * nw * 64 + lane];
      for (int v = 1; v < nw; ++v) t[x] += sums[((x * FJ + y) * nw + v) * 64 + lane];
    }
    const long long j = y * 16 + (lane & 15), i = i0 + 4 * (lane >> 4);
    const int left = j < g.nj && i < g.ni ? (int)(g.ni - i < 4 ? g.ni - i : 4) : 0;
    if (left > 0) {
      float v[4] = {t[0][0], t[0][1], t[0][2], t[0][3]};
      if constexpr (PAIR) {
        float u[4] = {t[1][0], t[1][1], t[1][2], t[1][3]};
        finish_pair<T>(g, i, j, left, v, u);
      } else {
        finish<T, O>(g, 0, i, j, left, v);
      }
    }
  }
  end_of_stores();
}

template <typename T, typename O, bool PAIR, int FJ>
hipError_t run(const GemmArgs &g, int waves, hipStream_t s) {
  hipLaunchKernelGGL((k_few<T, O, PAIR, FJ>), dim3((unsigned)((g.ni + 15) / 16)), dim3(64 * waves),
                     (PAIR ? 2 : 1) * FJ * waves * 1024, s, g);
  return hipGetLastError();
}

template <typename T, typename O, bool PAIR>
hipError_t run(const GemmArgs &g, int waves, hipStream_t s) {
  if (g.nj <= 16) return run<T, O, PAIR, 1>(g, waves, s);
  if (g.nj <= 32) return run<T, O, PAIR, 2>(g, waves, s);
  return run<T, O, PAIR, 4>(g, waves, s);
}

}  // namespace

bool few_sizes(const GemmArgs &g, const GemmForm &f) { return !f.a_trans && g.nj <= 64; }

hipError_t launch_few(const GemmArgs &g, const GemmForm &f, hipStream_t s) {
  // waves: as many as give each the same number of turns, up to 16 and 64 KB of sums
  const int unroll = g.nj <= 16 ? 8 : 4, fragments = (f.pair ? 2 : 1) * (g.nj <= 16 ? 1 : g.nj <= 32 ? 2 : 4);
  const int step = f.f32 ? 16 : 32, most = std::min(16, 64 / fragments);
  const int turns = std::max(1, (int)((g.nk + step * unroll - 1) / (step * unroll))), rounds = (turns + most - 1) / most;
  const int waves = (turns + rounds - 1) / rounds;
  if (f.pair) return f.f32 ? run<float, float, true>(g, waves, s) : run<bf16_t, bf16_t, true>(g, waves, s);
  if (f.f32) return run<float, float, false>(g, waves, s);
  return f.out_f32 ? run<bf16_t, float, false>(g, waves, s) : run<bf16_t, bf16_t, false>(g, waves, s);
}

// The forward products of up to 16 rows, as when sequences decode: every weight
// is read once, and its bytes are what counts.
//
// A workgroup takes 16 rows of the weights (with a pair 16 of each matrix), its
// waves take turns along k. The products run on the MFMA of 16 blocks of 4 x 4
// (v_mfma_f32_4x4x4_16b_bf16, 4x4x1 in fp32): lane l holds weight row and token
// l % 4 at the l / 4-th 16 bytes of k, so that a load instruction reads 256
// whole bytes of four rows, and each block sums its own part of k. (With the
// fragments of the 16 x 16 MFMA, lanes 0 to 15 of a load lie in 16 rows, and the
// vector cache takes them one at a time: 14.2 us for one token 9728 -> 2560,
// whose weights alone take 10 to read.) The 16 blocks are then added across the
// lanes, the waves in LDS, each in a fixed order. Rows and tokens past the end
// are read as the last one's, and their sums are not stored.
#include <algorithm>

#include "linear_dev.h"

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// 16 bytes of a row: eight bf16 or four fp32
typedef uint32_t Piece __attribute__((ext_vector_type(4)));
template <typename T>
__device__ __forceinline__ Piece piece(const T *p) {
  Piece v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
// n of its elements, the rest zero
template <typename T>
__device__ __forceinline__ Piece piece(const T *p, int n) {
  T e[16 / sizeof(T)] = {};
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(T); ++i)
    if (i < n) e[i] = p[i];
  Piece v;
  __builtin_memcpy(&v, e, 16);
  return v;
}
template <typename T>
__device__ __forceinline__ void mma(f32x4 &acc, Piece a, Piece b) {
  if constexpr (sizeof(T) == 2) {
    acc = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, u32x2_t{a[0], a[1]}),
                                                 __builtin_bit_cast(s16x4, u32x2_t{b[0], b[1]}), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, u32x2_t{a[2], a[3]}),
                                                 __builtin_bit_cast(s16x4, u32x2_t{b[2], b[3]}), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      acc = __builtin_amdgcn_mfma_f32_4x4x1f32(__uint_as_float(a[s]), __uint_as_float(b[s]), acc, 0, 0, 0);
  }
}

// x of the lane 4 further on (the lower four of each eight) and 4 back (the upper), by DPP.
__device__ __forceinline__ float from_xor4(float x) {
  const int v = __float_as_int(x);
  const int ahead = __builtin_amdgcn_update_dpp(0, v, 0x104, 0xf, 0xf, true);  // row_shl:4
  const int back = __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);   // row_shr:4
  return __int_as_float(threadIdx.x & 4 ? back : ahead);
}
__device__ __forceinline__ float from_xor8(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xf, 0xf, true));  // row_ror:8
}
// N values per lane, of each the sum over the lanes that agree in l % 4. A lane is left with N / 16 of them: at each
// step it keeps one half of its values (the upper one if the lane's bit is set) and gives the other half away. The
// swaps trade the upper lanes of one register for the lower ones of another, which is both at once.
template <int N, int BIT = 32>
__device__ __forceinline__ void scatter_sums(float (&v)[N]) {
  if constexpr (BIT >= 4) {
    const bool up = threadIdx.x & BIT;
    float h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (BIT >= 16) {
        const uint32_t lo = __float_as_uint(v[i]), hi = __float_as_uint(v[i + N / 2]);
        const auto r = BIT == 32 ? __builtin_amdgcn_permlane32_swap(lo, hi, false, false)
                                 : __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
        h[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
      } else {
        const float give = up ? v[i] : v[i + N / 2];
        h[i] = (up ? v[i + N / 2] : v[i]) + (BIT == 8 ? from_xor8(give) : from_xor4(give));
      }
    }
    scatter_sums<N / 2, BIT / 2>(h);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[i] = h[i];
  }
}

// Waves of a workgroup, at most, and steps loaded ahead: what gave the least of 1, 2 and 4 steps (8 tokens into the
// pair: 29.1, 25.6, 22.8 us; 16 tokens 9728 -> 2560: 20.1, 20.5, 24.3).
constexpr int kFewWaves = 8;
constexpr int few_steps(bool pair, int tq) { return tq == 4 ? 1 : pair && tq == 2 ? 4 : 2; }

template <typename T, typename O, bool PAIR, int TQ>
__global__ __launch_bounds__(64 * kFewWaves) void k_few(GemmArgs g) {
  constexpr int E = 16 / sizeof(T), STEP = 16 * E;  // k of a lane's piece, of a step
  constexpr int RQ = PAIR ? 8 : 4, U = few_steps(PAIR, TQ);
  constexpr int N = RQ * TQ * 4;
  __shared__ float sums[kFewWaves][N * 4];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const long long i0 = (long long)blockIdx.x * 16;
  const int nk = (int)g.nk, kl = (lane >> 2) * E;
  const T *a[RQ], *b[TQ];
#pragma unroll
  for (int x = 0; x < RQ; ++x) {
    const long long i = i0 + (x & 3) * 4 + (lane & 3);
    a[x] = reinterpret_cast<const T *>(g.a[x >> 2]) + (i < g.ni ? i : g.ni - 1) * g.lda + kl;
  }
#pragma unroll
  for (int y = 0; y < TQ; ++y) {
    const long long j = y * 4 + (lane & 3);
    b[y] = reinterpret_cast<const T *>(g.b[0]) + (j < g.nj ? j : g.nj - 1) * g.ldb + kl;
  }
  f32x4 acc[RQ][TQ];
#pragma unroll
  for (int x = 0; x < RQ; ++x)
#pragma unroll
    for (int y = 0; y < TQ; ++y) acc[x][y] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int full = nk / STEP;  // whole steps
  int s = w * U;
  for (; s + U <= full; s += nw * U) {
    Piece fa[U][RQ], fb[U][TQ];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int x = 0; x < RQ; ++x) fa[u][x] = piece(a[x] + (s + u) * STEP);
#pragma unroll
      for (int y = 0; y < TQ; ++y) fb[u][y] = piece(b[y] + (s + u) * STEP);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int x = 0; x < RQ; ++x)
#pragma unroll
        for (int y = 0; y < TQ; ++y) mma<T>(acc[x][y], fa[u][x], fb[u][y]);
  }
  // what is left of k, less than U steps and a part of one: the wave's whose turn it is
  for (; s < full + (nk % STEP != 0) && s / U % nw == w; ++s) {
    const int n = nk - s * STEP - kl;  // of this lane's piece
    Piece fa[RQ], fb[TQ];
#pragma unroll
    for (int x = 0; x < RQ; ++x) fa[x] = n >= E ? piece(a[x] + s * STEP) : piece(a[x] + s * STEP, n);
#pragma unroll
    for (int y = 0; y < TQ; ++y) fb[y] = n >= E ? piece(b[y] + s * STEP) : piece(b[y] + s * STEP, n);
#pragma unroll
    for (int x = 0; x < RQ; ++x)
#pragma unroll
      for (int y = 0; y < TQ; ++y) mma<T>(acc[x][y], fa[x], fb[y]);
  }
  float v[N];
#pragma unroll
  for (int x = 0; x < RQ; ++x)
#pragma unroll
    for (int y = 0; y < TQ; ++y)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[(x * TQ + y) * 4 + r] = acc[x][y][r];
  scatter_sums(v);
  const int at = (lane >> 5 & 1) * (N / 2) + (lane >> 4 & 1) * (N / 4) + (lane >> 3 & 1) * (N / 8) + (lane >> 2 & 1) * (N / 16);
#pragma unroll
  for (int i = 0; i < N / 16; ++i) sums[w][(at + i) * 4 + (lane & 3)] = v[i];
  __syncthreads();
  // four rows of one token per thread
  if (threadIdx.x >= 16 * TQ) return;
  const int c = threadIdx.x & 3, x = threadIdx.x >> 2 & 3, y = threadIdx.x >> 4;
  float t[2][4] = {};
#pragma unroll
  for (int h = 0; h < (PAIR ? 2 : 1); ++h)
    for (int u = 0; u < nw; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) t[h][r] += sums[u][(((h * 4 + x) * TQ + y) * 4 + r) * 4 + c];
  const long long j = y * 4 + c, i = i0 + x * 4;
  const int left = j < g.nj && i < g.ni ? (int)(g.ni - i < 4 ? g.ni - i : 4) : 0;
  if (left > 0) {
    if constexpr (PAIR)
      finish_pair<T>(g, i, j, left, t[0], t[1]);
    else
      finish<T, O>(g, 0, i, j, left, t[0]);
  }
  end_of_stores();
}

template <typename T, typename O, bool PAIR, int TQ>
hipError_t run(const GemmArgs &g, hipStream_t s) {
  // about 4096 waves (a pair's load twice as much), each with the same number of turns
  constexpr int U = few_steps(PAIR, TQ);
  const long long groups = (g.ni + 15) / 16;
  const int most = (int)std::max(2LL, std::min((long long)kFewWaves, (PAIR ? 2048 : 4096) / groups));
  const int step = 256 / (int)sizeof(T) * U, turns = std::max(1, (int)((g.nk + step - 1) / step));
  const int rounds = (turns + most - 1) / most, waves = (turns + rounds - 1) / rounds;
  hipLaunchKernelGGL((k_few<T, O, PAIR, TQ>), dim3((unsigned)groups), dim3(64 * waves), 0, s, g);
  return hipGetLastError();
}

template <typename T, typename O, bool PAIR>
hipError_t run(const GemmArgs &g, hipStream_t s) {
  if (g.nj <= 4) return run<T, O, PAIR, 1>(g, s);
  if (g.nj <= 8) return run<T, O, PAIR, 2>(g, s);
  return run<T, O, PAIR, 4>(g, s);
}

}  // namespace

// Up to 16 rows of tokens. Against the tiles that 17 rows take (with the call, some 11 us of host time at least): one to
// four tokens 9728 -> 2560 13.0 us and 17.2, eight 15.8, the pair 22.8 and 24.7; fp32 9728 -> 2560 32 to 37 and 40; odd
// widths 11.4 and 14 to 28. From 9 rows on large bf16 weights would gain by the tiles: 12 and 16 rows 18.0 and 19.5, the
// pair 29.2 and 30.0 (17.1 and 25.0). They stay here, where no call needs a workspace.
bool few_sizes(const GemmArgs &g, const GemmForm &f) { return !f.a_trans && g.nj <= 16; }

hipError_t launch_few(const GemmArgs &g, const GemmForm &f, hipStream_t s) {
  if (f.pair) return f.f32 ? run<float, float, true>(g, s) : run<bf16_t, bf16_t, true>(g, s);
  if (f.f32) return run<float, float, false>(g, s);
  return f.out_f32 ? run<bf16_t, float, false>(g, s) : run<bf16_t, bf16_t, false>(g, s);
}

// The matrix products of the plain layers: p = x W^T with bias, activation and
// residual, the two gated projections, and the products of their gradients.
//
// D[i][j] = sum_k A(i, k) B(j, k); the results lie in memory with i running
// fastest, so i is the weights' side (their rows forward, their columns
// backward) and j the tokens' (or, in a weight's gradient, its rows).
//
// MFMA 16x16 register layout (lane l, accumulator register r): A row i = l % 16
// and B row j = l % 16, with k = 8 (l / 16) .. +7 (bf16, 16x16x32) or k = l / 16
// (fp32, 16x16x4); D: j = l % 16, i = 4 (l / 16) + r.
#include <algorithm>
#include <cmath>

#include "grid.h"
#include "linear_dev.h"

namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// ---------------------------------------------------------------------------
// Any size, any alignment: tiles of 128 x 128, four waves of 64 x 64, staged
// through registers. fp32 products run on the fp32 MFMA, whose products and
// sums are those of fp32 FMAs.

constexpr int kTile = 128, kThreads = 256;

template <typename T>
constexpr int kBK = sizeof(T) == 2 ? 32 : 16;  // k per step: 64 bytes of a row

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

// One operand's tile: 128 rows of kBK, in LDS [row][k] where it lies by rows,
// [k][row] where it lies transposed.
template <typename T, bool TRANS>
struct Tile {
  static constexpr int BK = kBK<T>, PAD = 16 / (int)sizeof(T);
  static constexpr int PITCH = TRANS ? kTile + PAD : BK + PAD;
  static constexpr int SIZE = TRANS ? BK * PITCH : kTile * PITCH;
  static constexpr int N = kTile * BK / 8 / kThreads;
  Raw8<T> v[N];

  // row(r): the operand's row of tile row r, and its matrix in m; -1 if none
  template <class Row>
  __device__ __forceinline__ void load(const void *const (&m)[2], long long ld, long long row0, long long rows,
                                       long long k0, long long nk, Row &&row) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int q = threadIdx.x + n * kThreads;
      if constexpr (TRANS) {
        const long long k = k0 + q / (kTile / 8), r = row0 + q % (kTile / 8) * 8;
        v[n] = load_some(reinterpret_cast<const T *>(m[0]) + (k < nk ? k : 0) * ld + r, k < nk ? clamp8(rows - r) : 0);
      } else {
        int which = 0;
        const long long r = row(q / (BK / 8), which), k = k0 + q % (BK / 8) * 8;
        v[n] = load_some(reinterpret_cast<const T *>(m[which]) + (r < rows ? r : 0) * ld + k,
                         r < rows ? clamp8(nk - k) : 0);
      }
    }
  }
  __device__ __forceinline__ void put(T *lds) const {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int q = threadIdx.x + n * kThreads;
      const int at = TRANS ? q / (kTile / 8) * PITCH + q % (kTile / 8) * 8 : q / (BK / 8) * PITCH + q % (BK / 8) * 8;
      __builtin_memcpy(__builtin_assume_aligned(lds + at, 16), &v[n], sizeof v[n]);
    }
  }
};

// Fragment of rows r0 .. r0 + 15 of a step.
template <bool TRANS>
__device__ __forceinline__ bf16x8 fragment(const bf16_t *lds, int r0, int lane) {
  constexpr int P = Tile<bf16_t, TRANS>::PITCH;
  const int g = lane >> 4, t = lane & 15;
  if constexpr (TRANS) {
    // a transposing read takes, in each group of 16 lanes, a 4 x 16 block (lane t addresses row t/4, elements
    // 4(t%4) ..) and gives lane t column t of it
    const bf16_t *p = lds + (8 * g + (t >> 2)) * P + r0 + 4 * (t & 3);
    const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)p);
    const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)(p + 4 * P));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    return *reinterpret_cast<const bf16x8 *>(lds + (r0 + t) * P + 8 * g);
  }
}
// k = 4 (l / 16) + s in MFMA s of the step's four: the sum over k may take
// them in any order as long as A and B do alike.
template <bool TRANS>
__device__ __forceinline__ f32x4 fragment(const float *lds, int r0, int lane) {
  constexpr int P = Tile<float, TRANS>::PITCH;
  const int g = lane >> 4, t = lane & 15;
  if constexpr (TRANS) {
    f32x4 v;
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = lds[(4 * g + s) * P + r0 + t];
    return v;
  } else {
    return *reinterpret_cast<const f32x4 *>(lds + (r0 + t) * P + 4 * g);
  }
}
__device__ __forceinline__ void mma(f32x4 &acc, const bf16x8 &a, const bf16x8 &b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4 &acc, const f32x4 &a, const f32x4 &b) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], acc, 0, 0, 0);
}

// grid: i tiles (128 rows of A; with a pair 64 of each matrix), times j tiles, times batch, times splits of k
template <typename T, typename O, bool AT, bool BT, bool PAIR>
__global__ __launch_bounds__(kThreads, 2) void k_gemm(GemmArgs g, long long ti, long long tj, Parts parts) {
  using TA = Tile<T, AT>;
  using TB = Tile<T, BT>;
  __shared__ __attribute__((aligned(16))) T la[TA::SIZE];
  __shared__ __attribute__((aligned(16))) T lb[TB::SIZE];
  const long long n = group_index();
  if (n >= ti * tj * g.batch * parts.splits) return;
  const long long tile = n % (ti * tj);
  const int z = (int)(n / (ti * tj) % g.batch), split = (int)(n / (ti * tj * g.batch));
  const long long j0 = tile / ti * kTile, i0 = tile % ti * (PAIR ? kTile / 2 : kTile);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wi = w & 1, wj = w >> 1;
  f32x4 acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  // with a pair, a wave's 64 rows of A are 32 of the first matrix and the matching 32 of the second
  auto row_a = [&](int r, int &which) {
    if constexpr (PAIR) {
      which = (r >> 5) & 1;
      return i0 + (r >> 6) * 32 + (r & 31);
    }
    return i0 + r;
  };
  auto row_b = [&](int r, int &) { return j0 + r; };
  constexpr int BK = kBK<T>;
  const long long per = (g.nk + BK - 1) / BK, steps = per * g.segments;
  const long long first = steps * split / parts.splits, end = steps * (split + 1) / parts.splits;
  TA ta;
  TB tb;
  auto fetch = [&](long long st) {
    const int sg = st >= per;
    const long long k0 = (st - sg * per) * BK;
    const void *const a[2] = {PAIR ? g.a[0] : g.a[sg], g.a[1]};
    const void *const b[2] = {g.b[sg + z], nullptr};
    ta.load(a, g.lda, i0, g.ni, k0, g.nk, row_a);
    tb.load(b, g.ldb, j0, g.nj, k0, g.nk, row_b);
  };
  if (first < end) fetch(first);
  for (long long st = first; st < end; ++st) {
    ta.put(la);
    tb.put(lb);
    __syncthreads();
    if (st + 1 < end) fetch(st + 1);
    decltype(fragment<AT>(la, 0, 0)) fa[4], fb[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) fa[x] = fragment<AT>(la, wi * 64 + x * 16, lane);
#pragma unroll
    for (int x = 0; x < 4; ++x) fb[x] = fragment<BT>(lb, wj * 64 + x * 16, lane);
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) mma(acc[x][y], fa[x], fb[y]);
    __syncthreads();
  }
  if (parts.splits > 1) {
    float *p = parts.at + (n * kTile + wj * 64) * kTile + wi * 64;
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        *reinterpret_cast<f32x4 *>(p + (y * 16 + (lane & 15)) * kTile + x * 16 + 4 * (lane >> 4)) = acc[x][y];
    end_of_stores();
    return;
  }
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const long long j = j0 + wj * 64 + y * 16 + (lane & 15);
    if (j >= g.nj) continue;
#pragma unroll
    for (int x = 0; x < (PAIR ? 2 : 4); ++x) {
      const long long i = i0 + wi * (PAIR ? 32 : 64) + x * 16 + 4 * (lane >> 4);
      const int left = i < g.ni ? (int)(g.ni - i < 4 ? g.ni - i : 4) : 0;
      if (left == 0) continue;
      float v[4] = {acc[x][y][0], acc[x][y][1], acc[x][y][2], acc[x][y][3]};
      if constexpr (PAIR) {
        float u[4] = {acc[x + 2][y][0], acc[x + 2][y][1], acc[x + 2][y][2], acc[x + 2][y][3]};
        finish_pair<T>(g, i, j, left, v, u);
      } else {
        finish<T, O>(g, z, i, j, left, v);
      }
    }
  }
  end_of_stores();
}

// The splits' sums, added in their order, and what becomes of them. A thread
// takes eight elements i of one j of one tile.
template <typename T, typename O, bool PAIR>
__global__ __launch_bounds__(kThreads) void k_join(GemmArgs g, long long ti, long long tj, Parts parts) {
  const int wide = PAIR ? parts.ti / 2 : parts.ti;  // elements i of a tile
  const long long q = group_index() * kThreads + threadIdx.x, per = (long long)parts.tj * (wide / 8);
  const long long tiles = ti * tj * g.batch, n = q / per;
  if (n >= tiles) return;
  const int z = (int)(n / (ti * tj)), r = (int)(q % per), ii = r % (wide / 8) * 8, jj = r / (wide / 8);
  const long long tile = n % (ti * tj), i = tile % ti * wide + ii, j = tile / ti * parts.tj + jj;
  const int left = j < g.nj ? clamp8(g.ni - i) : 0;
  if (left == 0) return;
  const long long size = (long long)parts.ti * parts.tj;
  const float *p = parts.at + n * size + (long long)jj * parts.ti + (PAIR ? ii / parts.half * 2 * parts.half + ii % parts.half : ii);
  float v[8] = {}, u[8] = {};
  for (int s = 0; s < parts.splits; ++s) {
    float w[8];
    __builtin_memcpy(w, __builtin_assume_aligned(p, 16), 32);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += w[e];
    if constexpr (PAIR) {
      __builtin_memcpy(w, __builtin_assume_aligned(p + parts.half, 16), 32);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] += w[e];
    }
    p += tiles * size;
  }
  if constexpr (PAIR)
    finish_pair<T>(g, i, j, left, v, u);
  else
    finish<T, O>(g, z, i, j, left, v);
  end_of_stores();
}

template <typename T, typename O, bool AT, bool BT, bool PAIR>
hipError_t run_gemm(const GemmArgs &g, const GemmForm &f, int splits, hipStream_t s) {
  const long long ti = (g.ni + (PAIR ? kTile / 2 : kTile) - 1) / (PAIR ? kTile / 2 : kTile);
  const long long tj = (g.nj + kTile - 1) / kTile;
  if (ti * tj == 0) return hipSuccess;
  const Parts parts{(float *)g.ws, splits, kTile, kTile, kTile / 4};
  hipLaunchKernelGGL((k_gemm<T, O, AT, BT, PAIR>), group_grid(ti * tj * g.batch * splits), dim3(kThreads), 0, s, g, ti,
                     tj, parts);
  return splits > 1 ? launch_join(g, f, ti, tj, parts, s) : hipGetLastError();
}

template <typename T, typename O>
hipError_t run_gemm(const GemmArgs &g, const GemmForm &f, int splits, hipStream_t s) {
  if (f.pair) return run_gemm<T, T, false, false, true>(g, f, splits, s);
  if (!f.a_trans) return run_gemm<T, O, false, false, false>(g, f, splits, s);
  // gradients come in the operands' type
  return f.b_trans ? run_gemm<T, T, true, true, false>(g, f, splits, s)
                   : run_gemm<T, T, true, false, false>(g, f, splits, s);
}

// ---- the choice of tile and splits ----
//
// By what a launch would take: rounds of tiles over the device's 256 CUs times
// a tile's share of k, and for splits the fp32 sums written and read again and
// the second launch.

constexpr int kCus = 256;
struct Choice {
  int tile, splits;
  double us;
};

// us_slab: one tile's 64 of k with `slots` tiles at once on the device
Choice choose(const GemmArgs &g, const GemmForm &f, int tile, long long tiles, int slots, double us_slab) {
  Choice best{tile, 1, 1e30};
  const double slabs = (double)((g.nk + 63) / 64) * g.segments;
  const double bytes = (double)tiles * tile * tile * 4;
  for (int s = 1; s <= 32; ++s) {
    if (s > 1 && (slabs / s < 4 || bytes * s > 512e6)) break;
    const double rounds = (double)((tiles * s + slots - 1) / slots);
    double us = rounds * std::ceil(slabs / s) * us_slab;
    if (s > 1) us += 4.0 + 2.0 * bytes * s / 4.0e6;  // 4 TB/s
    if (us < 0.95 * best.us) best = Choice{tile, s, us};
  }
  return best;
}

long long general_tiles(const GemmArgs &g, const GemmForm &f) {
  const int wide = f.pair ? kTile / 2 : kTile;
  return (g.ni + wide - 1) / wide * ((g.nj + kTile - 1) / kTile) * g.batch;
}
Choice choose_general(const GemmArgs &g, const GemmForm &f) {
  return choose(g, f, kTile, general_tiles(g, f), 2 * kCus, f.f32 ? 10.5 : 1.7);
}
Choice choose_dense(const GemmArgs &g, const GemmForm &f) {
  const Choice big = choose(g, f, 256, dense_tiles(g, f, 256), kCus, 1.7);
  const Choice small = choose(g, f, 128, dense_tiles(g, f, 128), 2 * kCus, 1.1);
  return small.us < big.us ? small : big;
}
size_t parts_bytes(long long tiles, const Choice &c) {
  return c.splits > 1 ? (size_t)tiles * c.splits * c.tile * c.tile * 4 : 0;
}

// ---------------------------------------------------------------------------
// The gradient at the pre-activations, elementwise, and its sums over the rows
// for the biases. Without sums the arrays are taken as they lie, end to end.
// With sums a wave takes 512 columns (eight per lane) of every fourth row of a
// run; the waves' sums are added in LDS, the runs' by k_column_sums, each in a
// fixed order. Either way a thread loads all of a step before it stores any.

// Eight elements of the step from `at` on, `left` of them there.
template <typename D, typename T, bool GATED, bool NT>
struct ActStep {
  Raw8<D> dy;
  Raw8<T> p, u;
  template <typename V>
  static __device__ __forceinline__ Raw8<V> fetch(const void *base, long long at, int left) {
    const V *q = reinterpret_cast<const V *>(base) + at;
    if (!NT || left < 8) return load_some(q, left);
    Raw8<V> r;
    u32x4_any *to = reinterpret_cast<u32x4_any *>(&r);
    const u32x4_any *from = reinterpret_cast<const u32x4_any *>(q);
#pragma unroll
    for (int i = 0; i < (int)sizeof r / 16; ++i) to[i] = __builtin_nontemporal_load(from + i);
    return r;
  }
  static __device__ __forceinline__ void keep(void *base, long long at, int left, const float (&v)[8]) {
    T *q = reinterpret_cast<T *>(base) + at;
    if constexpr (NT && sizeof(T) == 2) {
      if (left >= 8) {
        stream_w(q, true, v);
        end_of_stores();
        return;
      }
    }
    put(q, left, v);
  }
  __device__ __forceinline__ void load(const ActGradArgs &a, long long at, int left) {
    dy = fetch<D>(a.dy, at, left);
    if (GATED || a.p) p = fetch<T>(a.p, at, left);
    if constexpr (GATED) u = fetch<T>(a.u, at, left);
  }
  // q, and with a pair also q2, rounded and kept
  __device__ __forceinline__ void apply(const ActGradArgs &a, long long at, int left, float (&q)[8], float (&q2)[8]) const {
    float d[8], x[8], y[8];
    expand(dy, d);
    if constexpr (GATED) {
      expand(p, x);
      expand(u, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float f, df;
        act_grad_of(x[e], a.act, f, df);
        q[e] = d[e] * y[e] * df;
        q2[e] = d[e] * f;
      }
      keep(a.out2, at, left, q2);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = a.scale * d[e];
      if (a.p) {
        expand(p, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float f, df;
          act_grad_of(x[e], a.act, f, df);
          q[e] *= df;
        }
      }
    }
    if (a.out) keep(a.out, at, left, q);
  }
};

constexpr int kFlat = 2;  // steps of a thread
template <typename D, typename T, bool GATED, bool NT>
__global__ __launch_bounds__(kThreads) void k_act_grad(ActGradArgs a) {
  const long long n = a.rows * a.n, at = (group_index() * kFlat * kThreads + threadIdx.x) * 8;
  ActStep<D, T, GATED, NT> st[kFlat];
#pragma unroll
  for (int k = 0; k < kFlat; ++k) st[k].load(a, at + k * kThreads * 8, clamp8(n - at - k * kThreads * 8));
#pragma unroll
  for (int k = 0; k < kFlat; ++k) {
    float q[8], q2[8];
    st[k].apply(a, at + k * kThreads * 8, clamp8(n - at - k * kThreads * 8), q, q2);
  }
  end_of_stores();
}

constexpr int kWaveCols = 512, kSumWaves = kThreads / 64;
// runs of rows: enough workgroups to fill the device, of at least four rows per wave
long long row_runs(long long rows, long long n) {
  const long long groups = (n + kWaveCols - 1) / kWaveCols;
  return std::max(1LL, std::min((rows + 4 * kSumWaves - 1) / (4 * kSumWaves), (2048 + groups - 1) / groups));
}

template <typename D, typename T, bool GATED, bool NT>
__global__ __launch_bounds__(kThreads) void k_act_grad_sums(ActGradArgs a, long long runs) {
  __shared__ __attribute__((aligned(16))) float red[kSumWaves][GATED ? 2 : 1][kWaveCols];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const long long c = (long long)blockIdx.x * kWaveCols + lane * 8;
  const int left = clamp8(a.n - c);
  const long long run = blockIdx.y, r1 = a.rows * (run + 1) / runs;
  float s1[8] = {}, s2[8] = {};
  for (long long r = a.rows * run / runs + w; r < r1; r += 2 * kSumWaves) {
    ActStep<D, T, GATED, NT> st[2];
    const bool two = r + kSumWaves < r1;
    st[0].load(a, r * a.n + c, left);
    st[1].load(a, (two ? r + kSumWaves : r) * a.n + c, two ? left : 0);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 1 && !two) break;
      float q[8], q2[8];
      st[k].apply(a, (r + k * kSumWaves) * a.n + c, left, q, q2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s1[e] += q[e];
        if constexpr (GATED) s2[e] += q2[e];
      }
    }
  }
  __builtin_memcpy(&red[w][0][lane * 8], s1, 32);
  if constexpr (GATED) __builtin_memcpy(&red[w][1][lane * 8], s2, 32);
  __syncthreads();
  for (int i = threadIdx.x; i < kWaveCols * (GATED ? 2 : 1); i += kThreads) {
    const int half = i / kWaveCols, k = i % kWaveCols;
    const long long col = (long long)blockIdx.x * kWaveCols + k;
    if (col >= a.n) continue;
    float s = red[0][half][k];
#pragma unroll
    for (int v = 1; v < kSumWaves; ++v) s += red[v][half][k];
    a.part[(half * runs + run) * a.n + col] = s;
  }
}

// A workgroup adds the runs of 64 columns, a wave every sixteenth.
__global__ __launch_bounds__(1024) void k_column_sums(const float *part, long long runs, long long n, float *sum,
                                                      float *sum2, int accumulate) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const long long c = (long long)blockIdx.x * 64 + lane;
  const float *p = part + blockIdx.y * runs * n + c;
  float s = 0.f;
  if (c < n) {
#pragma unroll 4
    for (long long r = w; r < runs; r += 16) s += p[r * n];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w != 0 || c >= n) return;
#pragma unroll
  for (int v = 1; v < 16; ++v) s += red[v][lane];
  float *out = blockIdx.y ? sum2 : sum;
  out[c] = accumulate ? out[c] + s : s;
}

// arrays of more bytes than this are read and written past the caches, of which the last level holds 256 MiB
constexpr long long kStreamBytes = 512LL << 20;

template <typename D, typename T, bool GATED, bool NT>
hipError_t run_act_grad(const ActGradArgs &a, hipStream_t s) {
  if (!a.sum) {
    const long long groups = (a.rows * a.n + kFlat * kThreads * 8 - 1) / (kFlat * kThreads * 8);
    if (groups > 0) hipLaunchKernelGGL((k_act_grad<D, T, GATED, NT>), group_grid(groups), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  const long long runs = row_runs(a.rows, a.n);
  hipLaunchKernelGGL((k_act_grad_sums<D, T, GATED, NT>),
                     dim3((unsigned)((a.n + kWaveCols - 1) / kWaveCols), (unsigned)runs), dim3(kThreads), 0, s, a, runs);
  hipLaunchKernelGGL(k_column_sums, dim3((unsigned)((a.n + 63) / 64), GATED ? 2 : 1), dim3(1024), 0, s, a.part, runs,
                     a.n, a.sum, a.sum2, a.accumulate);
  return hipGetLastError();
}

template <typename D, typename T>
hipError_t run_act_grad(const ActGradArgs &a, hipStream_t s) {
  const bool nt = a.rows * a.n * (long long)(sizeof(D) + (a.u ? 4 : a.p ? 2 : 1) * sizeof(T)) > kStreamBytes;
  if (a.u) return nt ? run_act_grad<D, T, true, true>(a, s) : run_act_grad<D, T, true, false>(a, s);
  return nt ? run_act_grad<D, T, false, true>(a, s) : run_act_grad<D, T, false, false>(a, s);
}

template <typename T, typename O>
hipError_t run_join(const GemmArgs &g, bool pair, long long ti, long long tj, const Parts &p, hipStream_t s) {
  const long long threads = ti * tj * g.batch * p.tj * ((pair ? p.ti / 2 : p.ti) / 8);
  const dim3 grid = group_grid((threads + kThreads - 1) / kThreads);
  if (pair)
    hipLaunchKernelGGL((k_join<T, T, true>), grid, dim3(kThreads), 0, s, g, ti, tj, p);
  else
    hipLaunchKernelGGL((k_join<T, O, false>), grid, dim3(kThreads), 0, s, g, ti, tj, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_join(const GemmArgs &g, const GemmForm &f, long long ti, long long tj, const Parts &p, hipStream_t s) {
  if (f.f32) return run_join<float, float>(g, f.pair, ti, tj, p, s);
  return f.out_f32 ? run_join<bf16_t, float>(g, f.pair, ti, tj, p, s) : run_join<bf16_t, bf16_t>(g, f.pair, ti, tj, p, s);
}

size_t gemm_ws_bytes(const GemmArgs &g, const GemmForm &f) {
  if (few_sizes(g, f)) return 0;
  const size_t general = parts_bytes(general_tiles(g, f), choose_general(g, f));
  if (!dense_sizes(g, f)) return general;
  const Choice c = choose_dense(g, f);
  return std::max(general, parts_bytes(dense_tiles(g, f, c.tile), c));
}

hipError_t launch_gemm(const GemmArgs &g, const GemmForm &f, hipStream_t s) {
  if (few_sizes(g, f)) return launch_few(g, f, s);
  if (dense_sizes(g, f) && dense_aligned(g, f)) {
    const Choice c = choose_dense(g, f);
    return launch_dense(g, f, c.tile, c.splits, s);
  }
  const int splits = choose_general(g, f).splits;
  if (f.f32) return run_gemm<float, float>(g, f, splits, s);
  return f.out_f32 ? run_gemm<bf16_t, float>(g, f, splits, s) : run_gemm<bf16_t, bf16_t>(g, f, splits, s);
}

size_t act_grad_ws_bytes(long long rows, long long n, bool gated) {
  return (size_t)row_runs(rows, n) * n * 4 * (gated ? 2 : 1);
}

hipError_t launch_act_grad(const ActGradArgs &a, hipStream_t s) {
  if (a.f32) return run_act_grad<float, float>(a, s);
  return a.dy_f32 ? run_act_grad<float, bf16_t>(a, s) : run_act_grad<bf16_t, bf16_t>(a, s);
}

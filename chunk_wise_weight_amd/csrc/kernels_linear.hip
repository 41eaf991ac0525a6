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
#include "tiles.h"

namespace {

// ---------------------------------------------------------------------------
// Any size, any alignment: tiles of 128 x 128 (four waves of 64 x 64) or 64 x 64
// (of 32 x 32), staged through registers into two LDS buffers in turn. The
// loads of step n + 2 are issued when step n's registers have gone to LDS. fp32
// products run on the fp32 MFMA, whose products and sums are those of fp32
// FMAs. Measured: 4099 x 1021 x 2047 in bf16 53 us, 320 TFLOP/s, bound by the
// waits for its loads (8192 x 1021 x 4095 157 us, 104 with rows copied and tiles
// that go straight to LDS); in fp32 181 us, 95 TFLOP/s.

constexpr int kThreads = 256, BK = 32;  // k per step

// One operand's tile: ROWS rows of 32 k, in LDS [row][k] where it lies by rows, [k][row] where it lies transposed.
template <typename T, bool TRANS, int ROWS>
struct Tile {
  static constexpr int PAD = 16 / (int)sizeof(T), PITCH = (TRANS ? ROWS : BK) + PAD;
  static constexpr int SIZE = (TRANS ? BK : ROWS) * PITCH;
  static constexpr int ACROSS = (TRANS ? ROWS : BK) / 8;  // pieces of eight to a line
  static constexpr int N = ROWS * BK / 8 / kThreads;
  Raw8<T> v[N];

  // row(r): the operand's row of tile row r, and its matrix in m
  template <class Row>
  __device__ __forceinline__ void load(const void *const (&m)[2], long long ld, long long row0, long long rows,
                                       long long k0, long long nk, Row &&row) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int q = threadIdx.x + n * kThreads;
      if constexpr (TRANS) {
        const long long k = k0 + q / ACROSS, r = row0 + q % ACROSS * 8;
        v[n] = load_some(reinterpret_cast<const T *>(m[0]) + (k < nk ? k : 0) * ld + r, k < nk ? clamp8(rows - r) : 0);
      } else {
        int which = 0;
        const long long r = row(q / ACROSS, which), k = k0 + q % ACROSS * 8;
        v[n] = load_some(reinterpret_cast<const T *>(m[which]) + (r < rows ? r : 0) * ld + k,
                         r < rows ? clamp8(nk - k) : 0);
      }
    }
  }
  __device__ __forceinline__ void put(T *lds) const {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int q = threadIdx.x + n * kThreads;
      __builtin_memcpy(__builtin_assume_aligned(lds + q / ACROSS * PITCH + q % ACROSS * 8, 16), &v[n], sizeof v[n]);
    }
  }
};

// Fragment of rows r0 .. r0 + 15 of a step.
template <bool TRANS, int P>
__device__ __forceinline__ bf16x8 fragment(const bf16_t *lds, int r0, int lane) {
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
// k = 16 h + 4 (l / 16) + s in MFMA 4 h + s of the step's eight: the sum over k may take them in any order as long as A
// and B do alike.
struct Fragment32 {
  f32x4 h[2];
};
template <bool TRANS, int P>
__device__ __forceinline__ Fragment32 fragment(const float *lds, int r0, int lane) {
  const int g = lane >> 4, t = lane & 15;
  Fragment32 v;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (TRANS) {
#pragma unroll
      for (int s = 0; s < 4; ++s) v.h[h][s] = lds[(16 * h + 4 * g + s) * P + r0 + t];
    } else {
      v.h[h] = *reinterpret_cast<const f32x4 *>(lds + (r0 + t) * P + 16 * h + 4 * g);
    }
  }
  return v;
}
// A step's products. The fp32 ones that add to one sum are F apart: one directly behind the other would wait for it.
template <int F>
__device__ __forceinline__ void multiply(f32x4 (&acc)[F][F], const bf16x8 (&a)[F], const bf16x8 (&b)[F]) {
#pragma unroll
  for (int x = 0; x < F; ++x)
#pragma unroll
    for (int y = 0; y < F; ++y) acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[x], b[y], acc[x][y], 0, 0, 0);
}
template <int F>
__device__ __forceinline__ void multiply(f32x4 (&acc)[F][F], const Fragment32 (&a)[F], const Fragment32 (&b)[F]) {
#pragma unroll
  for (int x = 0; x < F; ++x)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int y = 0; y < F; ++y)
          acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[x].h[h][s], b[y].h[h][s], acc[x][y], 0, 0, 0);
}

// grid: i tiles (TILE rows of A; with a pair half as many of each matrix), times j tiles, times batch, times splits of k
template <typename T, typename O, bool AT, bool BT, bool PAIR, int TILE>
__global__ __launch_bounds__(kThreads, 2) void k_gemm(GemmArgs g, long long ti, long long tj, Parts parts) {
  using TA = Tile<T, AT, TILE>;
  using TB = Tile<T, BT, TILE>;
  constexpr int F = TILE / 32, HALF = TILE / 4;  // fragments of a wave either way; a pair's rows of one matrix in a wave
  __shared__ __attribute__((aligned(16))) T lds[2][TA::SIZE + TB::SIZE];
  const long long n = group_index();
  if (n >= ti * tj * g.batch * parts.splits) return;
  const long long tile = n % (ti * tj);
  const int z = (int)(n / (ti * tj) % g.batch), split = (int)(n / (ti * tj * g.batch));
  const long long j0 = tile / ti * TILE, i0 = tile % ti * (PAIR ? TILE / 2 : TILE);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wi = w & 1, wj = w >> 1;
  f32x4 acc[F][F];
#pragma unroll
  for (int a = 0; a < F; ++a)
#pragma unroll
    for (int b = 0; b < F; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  // with a pair, a wave's rows of A are HALF of the first matrix and the matching HALF of the second
  auto row_a = [&](int r, int &which) {
    if constexpr (PAIR) {
      which = r / HALF & 1;
      return i0 + r / (2 * HALF) * HALF + r % HALF;
    }
    return i0 + r;
  };
  auto row_b = [&](int r, int &) { return j0 + r; };
  const long long per = (g.nk + BK - 1) / BK, steps = per * g.segments;
  const long long first = steps * split / parts.splits, end = steps * (split + 1) / parts.splits;
  TA ta[2];
  TB tb[2];
  auto fetch = [&](long long st, TA &a, TB &b) {
    const int sg = st >= per;
    const long long k0 = (st - sg * per) * BK;
    const void *const pa[2] = {PAIR ? g.a[0] : g.a[sg], g.a[1]};
    const void *const pb[2] = {g.b[sg + z], nullptr};
    a.load(pa, g.lda, i0, g.ni, k0, g.nk, row_a);
    b.load(pb, g.ldb, j0, g.nj, k0, g.nk, row_b);
  };
  // A wave that writes a buffer has passed the barrier of the step between, which every wave reaches only after its
  // reads of that buffer.
  auto step = [&](long long st, TA &a, TB &b, T *buf) {
    T *la = buf, *lb = buf + TA::SIZE;
    a.put(la);
    b.put(lb);
    if (st + 2 < end) fetch(st + 2, a, b);
    __syncthreads();
    decltype(fragment<AT, TA::PITCH>(la, 0, 0)) fa[F], fb[F];
#pragma unroll
    for (int x = 0; x < F; ++x) fa[x] = fragment<AT, TA::PITCH>(la, (wi * F + x) * 16, lane);
#pragma unroll
    for (int x = 0; x < F; ++x) fb[x] = fragment<BT, TB::PITCH>(lb, (wj * F + x) * 16, lane);
    multiply(acc, fa, fb);
  };
  if (first < end) fetch(first, ta[0], tb[0]);
  if (first + 1 < end) fetch(first + 1, ta[1], tb[1]);
  for (long long st = first; st < end; st += 2) {
    step(st, ta[0], tb[0], lds[0]);
    if (st + 1 < end) step(st + 1, ta[1], tb[1], lds[1]);
  }
  if (parts.splits > 1) {
    float *p = parts.at + (n * TILE + wj * (TILE / 2)) * TILE + wi * (TILE / 2);
#pragma unroll
    for (int y = 0; y < F; ++y)
#pragma unroll
      for (int x = 0; x < F; ++x)
        *reinterpret_cast<f32x4 *>(p + (y * 16 + (lane & 15)) * TILE + x * 16 + 4 * (lane >> 4)) = acc[x][y];
    end_of_stores();
    return;
  }
#pragma unroll
  for (int y = 0; y < F; ++y) {
    const long long j = j0 + (wj * F + y) * 16 + (lane & 15);
    if (j >= g.nj) continue;
#pragma unroll
    for (int x = 0; x < (PAIR ? F / 2 : F); ++x) {
      const long long i = i0 + wi * (PAIR ? HALF : 2 * HALF) + x * 16 + 4 * (lane >> 4);
      const int left = i < g.ni ? (int)(g.ni - i < 4 ? g.ni - i : 4) : 0;
      if (left == 0) continue;
      float v[4] = {acc[x][y][0], acc[x][y][1], acc[x][y][2], acc[x][y][3]};
      if constexpr (PAIR) {
        float u[4] = {acc[x + F / 2][y][0], acc[x + F / 2][y][1], acc[x + F / 2][y][2], acc[x + F / 2][y][3]};
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

// ---------------------------------------------------------------------------
// Rows copied to where they start on 16 bytes, zero behind their ends, so that
// a product of odd widths can run on the tiles that load whole pieces (12.6 MB:
// 10.6 us, half of it a launch and its ramp).

struct PackJob {
  const void *src;
  void *dst;
  long long rows, n, first;  // first: pieces of eight before this job's
};
struct PackJobs {
  PackJob job[4];
  int count;
  long long pieces;
};
template <typename T>
__global__ __launch_bounds__(kThreads) void k_pack(PackJobs p) {
  const long long q = group_index() * kThreads + threadIdx.x;
  if (q >= p.pieces) return;
  int k = 0;
#pragma unroll
  for (int i = 1; i < 4; ++i)
    if (i < p.count && q >= p.job[i].first) k = i;
  const long long n = p.job[k].n, per = (n + 7) / 8, at = q - p.job[k].first, r = at / per, c = at % per * 8;
  const Raw8<T> v = load_some((const T *)p.job[k].src + r * n + c, clamp8(n - c));
  __builtin_memcpy(__builtin_assume_aligned((T *)p.job[k].dst + at * 8, 16), &v, sizeof v);
  end_of_stores();
}

long long pad8(long long n) { return (n + 7) / 8 * 8; }

// ---- the choice of kernel, tile and splits ----
//
// By what a launch would take: its 64-k slabs times what the tiles take for one
// slab (us_slab, per form); for splits the fp32 sums written and read again, in
// the last-level cache up to 100 MB, and the second launch; for rows that are
// copied first their bytes and a launch. The times are measured ones
// (microseconds). Over 38 products of 17 to 20000 rows of all forms and both
// types the choice took at most 7 % more than the best of both kernels' tiles
// with 1 to 12 splits. The general kernel's bf16 shares are those of odd rows:
// with lower ones (0.9 and 0.42) gradients of odd widths were not copied that
// gain by it (20000 x 513 x 1365 257 us, 163 with the copy). They serve rows of
// whole pieces alike, which come here where an array does not start on 16
// bytes: over 16 of those it took at most 9 % more than the best (with the lower
// ones up to 30: dx of 8192 x 1024 x 4096 181 us, 139).

constexpr int kCus = 256;
struct Choice {
  int tile, splits;
  double us;
};

// us_slab(n): of n tiles on the device; us_once: what else they take when they are not split
template <class F>
Choice choose(const GemmArgs &g, int tile, long long tiles, F &&us_slab, double us_once = 0) {
  Choice best{tile, 1, 1e30};
  const double slabs = (double)((g.nk + 63) / 64) * g.segments;
  const double bytes = (double)tiles * tile * tile * 4;
  for (int s = 1; s <= 32; ++s) {
    if (s > 1 && (slabs / s < 4 || bytes * s > 512e6)) break;
    double us = std::ceil(slabs / s) * us_slab(tiles * s);
    us += s == 1 ? us_once : 5.0 + 2.0 * bytes * s / (bytes * s <= 100e6 ? 6.0e6 : 4.0e6);
    if (us < 0.97 * best.us) best = Choice{tile, s, us};
  }
  return best;
}

long long general_tiles(const GemmArgs &g, const GemmForm &f, int tile) {
  const int wide = f.pair ? tile / 2 : tile;
  return (g.ni + wide - 1) / wide * ((g.nj + tile - 1) / tile) * g.batch;
}
// Several tiles share a CU: what one takes by itself, or each one's share on the fullest CU.
auto shared(double alone, double share) {
  return [=](long long n) { return std::max(alone, (double)((n + kCus - 1) / kCus) * share); };
}
Choice choose_general(const GemmArgs &g, const GemmForm &f) {
  const double wait = f.b_trans ? 3.5 : f.a_trans ? 2.6 : 1.8;  // bf16, a tile of 128 alone
  const Choice big = choose(g, 128, general_tiles(g, f, 128), shared(f.f32 ? 5.1 : wait, f.f32 ? 4.4 : 1.5));
  const Choice small = choose(g, 64, general_tiles(g, f, 64), shared(f.f32 ? 2.2 : 0.5 * wait, f.f32 ? 1.17 : 0.6));
  return small.us < big.us ? small : big;
}
// Here bf16 tiles of 256 run in rounds of one per CU and those of 128 in rounds of two; the others share as above.
Choice choose_dense(const GemmArgs &g, const GemmForm &f) {
  auto pairs = [](long long n) {
    const double rest = (double)(n % (2 * kCus)) / kCus;
    return 1.2 * (n / (2 * kCus)) + (rest > 0 ? 0.9 + 0.3 * std::max(0.0, rest - 1) : 0);
  };
  const long long mid = dense_tiles(g, f, 128), small = dense_tiles(g, f, 64);
  Choice best = f.f32 ? choose(g, 128, mid, shared(4.4, 3.97)) : choose(g, 128, mid, pairs);
  const Choice s = choose(g, 64, small, f.f32 ? shared(1.45, 1.03) : shared(0.34, 0.25));
  if (s.us < best.us) best = s;
  if (f.f32) return best;  // four fp32 tiles of 128 take what one of 256 does
  // A tile of 256 stores by itself on its CU, and odd rows of results take it 7 us longer where there is a bias (4099 x 1021
  // x 2047 with bias and GELU: 56 us, with tiles of 128 51, of 64 47; 8192 x 1024 x 4095: 87, 98, 123). Without one it takes
  // less: 44 us against 45 and 45 (fp32 results 44, 55, 50), and the rule, which knows sizes alone, then takes those.
  const long long n = dense_tiles(g, f, 256);
  const Choice b = choose(g, 256, n, shared(1.75, 1.75), g.ldo % 8 ? 7.0 * ((n + kCus - 1) / kCus) : 0);
  return best.us < b.us ? best : b;
}
size_t parts_bytes(long long tiles, const Choice &c) {
  return c.splits > 1 ? (size_t)tiles * c.splits * c.tile * c.tile * 4 : 0;
}

// How a product runs, by its sizes: which operands are copied first, and the workspace: copies, then sums.
struct Plan {
  bool dense, pack_a, pack_b;
  Choice choice;
  GemmArgs g;  // sizes as they are after the copies
  long long rows_a, rows_b;
  int count_a, count_b;  // matrices of each operand
  size_t copies, parts;
};
Plan plan_of(const GemmArgs &g, const GemmForm &f) {
  Plan p{};
  p.g = g;
  p.choice = choose_general(g, f);
  p.parts = parts_bytes(general_tiles(g, f, p.choice.tile), p.choice);
  Plan d = p;
  d.dense = true;
  d.pack_a = g.lda % (f.f32 ? 4 : 8) != 0;
  d.pack_b = g.ldb % (f.f32 ? 4 : 8) != 0;
  if (d.pack_a) d.g.lda = pad8(g.lda);
  if (d.pack_b) d.g.ldb = pad8(g.ldb);
  d.rows_a = f.a_trans ? g.nk : g.ni;
  d.rows_b = f.b_trans ? g.nk : g.nj;
  d.count_a = f.pair || g.segments > 1 ? 2 : 1;
  d.count_b = g.segments > 1 || g.batch > 1 ? 2 : 1;
  if (!dense_sizes(d.g, f)) return p;
  d.choice = choose_dense(g, f);
  d.parts = parts_bytes(dense_tiles(g, f, d.choice.tile), d.choice);
  if (d.pack_a) d.copies += (size_t)d.count_a * d.rows_a * d.g.lda * (f.f32 ? 4 : 2);
  if (d.pack_b) d.copies += (size_t)d.count_b * d.rows_b * d.g.ldb * (f.f32 ? 4 : 2);
  const double us = d.choice.us + (d.copies ? 4.0 + 2.0 * d.copies / 4.0e6 : 0.0);
  return d.copies && us >= p.choice.us ? p : d;
}

template <typename T, typename O, bool AT, bool BT, bool PAIR, int TILE>
hipError_t run_gemm(const GemmArgs &g, const GemmForm &f, int splits, hipStream_t s) {
  const int wide = PAIR ? TILE / 2 : TILE;
  const long long ti = (g.ni + wide - 1) / wide, tj = (g.nj + TILE - 1) / TILE;
  if (ti * tj == 0) return hipSuccess;
  const Parts parts{(float *)g.ws, splits, TILE, TILE, TILE / 4};
  hipLaunchKernelGGL((k_gemm<T, O, AT, BT, PAIR, TILE>), group_grid(ti * tj * g.batch * splits), dim3(kThreads), 0, s,
                     g, ti, tj, parts);
  return splits > 1 ? launch_join(g, f, ti, tj, parts, s) : hipGetLastError();
}
template <typename T, typename O, bool AT, bool BT, bool PAIR>
hipError_t run_gemm(const GemmArgs &g, const GemmForm &f, const Choice &c, hipStream_t s) {
  return c.tile == 128 ? run_gemm<T, O, AT, BT, PAIR, 128>(g, f, c.splits, s)
                       : run_gemm<T, O, AT, BT, PAIR, 64>(g, f, c.splits, s);
}
template <typename T, typename O>
hipError_t run_gemm(const GemmArgs &g, const GemmForm &f, const Choice &c, hipStream_t s) {
  if (f.pair) return run_gemm<T, T, false, false, true>(g, f, c, s);
  if (!f.a_trans) return run_gemm<T, O, false, false, false>(g, f, c, s);
  // gradients come in the operands' type
  return f.b_trans ? run_gemm<T, T, true, true, false>(g, f, c, s) : run_gemm<T, T, true, false, false>(g, f, c, s);
}

// ---------------------------------------------------------------------------
// The gradient at the pre-activations, elementwise, and its sums over the rows
// for the biases. It is rounded once to the type of the products' operands: in
// bf16 that is what their MFMA takes, and the one rounding beside those of the
// results (their error grows by 1.41; two bf16 parts of it would keep 16 bits and
// double the products, 5.1 of 5.65 ms for a pair of 32768 x 2560 x 9728). The
// sums take the unrounded ones. Without sums the arrays are taken as they lie, end to end.
// With sums, or where rows are set apart, a wave takes 512 columns (eight per
// lane) of every fourth row of a run; the waves' sums are added in LDS, the
// runs' by k_column_sums, each in a fixed order. Either way a thread loads all
// of a step before it stores any. Bound by memory: 32768 x 9728 of a pair 556 us,
// 5.7 TB/s; 8192 x 4096 with sums 41 us, 4.9 TB/s, and 4.7 us to add them.

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
  // pad: a short run becomes a whole one
  static __device__ __forceinline__ void keep(void *base, long long at, int left, bool pad, float (&v)[8]) {
    if (pad && left < 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < left ? v[e] : 0.f;
      if (left > 0) left = 8;
    }
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
  // q, and with a pair also q2, rounded and kept at `to`
  __device__ __forceinline__ void apply(const ActGradArgs &a, long long to, int left, float (&q)[8], float (&q2)[8]) const {
    const bool pad = a.ldo > a.n;
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
      keep(a.out2, to, left, pad, q2);
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
    if (a.out) keep(a.out, to, left, pad, q);
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
      st[k].apply(a, (r + k * kSumWaves) * a.ldo + c, left, q, q2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s1[e] += q[e];
        if constexpr (GATED) s2[e] += q2[e];
      }
    }
  }
  if (!a.sum) {
    end_of_stores();
    return;
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
  if (!a.sum && a.ldo == a.n) {
    const long long groups = (a.rows * a.n + kFlat * kThreads * 8 - 1) / (kFlat * kThreads * 8);
    if (groups > 0) hipLaunchKernelGGL((k_act_grad<D, T, GATED, NT>), group_grid(groups), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  const long long runs = row_runs(a.rows, a.n);
  hipLaunchKernelGGL((k_act_grad_sums<D, T, GATED, NT>),
                     dim3((unsigned)((a.n + kWaveCols - 1) / kWaveCols), (unsigned)runs), dim3(kThreads), 0, s, a, runs);
  if (!a.sum) return hipGetLastError();
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
  // operands that need no copy may still not start on 16 bytes, and the product then runs as a general one
  const Choice c = choose_general(g, f);
  const Plan p = plan_of(g, f);
  return std::max(parts_bytes(general_tiles(g, f, c.tile), c), p.copies + p.parts);
}

GemmPlan gemm_plan(const GemmArgs &g, const GemmForm &f) {
  if (few_sizes(g, f)) return GemmPlan{TTT_KERNEL_FEW, 0, 1, 0};
  const Plan p = plan_of(g, f);
  const int copies = p.dense ? (p.pack_a ? p.count_a : 0) + (p.pack_b ? p.count_b : 0) : 0;
  return GemmPlan{p.dense ? TTT_KERNEL_DIRECT : TTT_KERNEL_GENERAL, p.choice.tile, p.choice.splits, copies};
}

hipError_t launch_gemm(const GemmArgs &g, const GemmForm &f, hipStream_t s) {
  if (few_sizes(g, f)) return launch_few(g, f, s);
  const Plan p = plan_of(g, f);
  uintptr_t low = 0;
  for (int i = 0; i < p.count_a; ++i) low |= p.pack_a ? 0 : (uintptr_t)g.a[i];
  for (int i = 0; i < p.count_b; ++i) low |= p.pack_b ? 0 : (uintptr_t)g.b[i];
  if (p.dense && low % 16 == 0) {
    GemmArgs d = p.g;
    if (p.copies) {
      PackJobs jobs{};
      char *to = (char *)g.ws;
      auto add = [&](const void *&m, long long rows, long long n) {
        jobs.job[jobs.count++] = PackJob{m, to, rows, n, jobs.pieces};
        m = to;
        to += rows * pad8(n) * (f.f32 ? 4 : 2);
        jobs.pieces += rows * (pad8(n) / 8);
      };
      for (int i = 0; p.pack_a && i < p.count_a; ++i) add(d.a[i], p.rows_a, g.lda);
      for (int i = 0; p.pack_b && i < p.count_b; ++i) add(d.b[i], p.rows_b, g.ldb);
      hipLaunchKernelGGL(f.f32 ? k_pack<float> : k_pack<bf16_t>, group_grid((jobs.pieces + kThreads - 1) / kThreads),
                         dim3(kThreads), 0, s, jobs);
      d.ws = to;
    }
    return launch_dense(d, f, p.choice.tile, p.choice.splits, s);
  }
  const Choice c = choose_general(g, f);
  if (f.f32) return run_gemm<float, float>(g, f, c, s);
  return f.out_f32 ? run_gemm<bf16_t, float>(g, f, c, s) : run_gemm<bf16_t, bf16_t>(g, f, c, s);
}

size_t act_grad_ws_bytes(long long rows, long long n, bool gated) {
  return (size_t)row_runs(rows, n) * n * 4 * (gated ? 2 : 1);
}

hipError_t launch_act_grad(const ActGradArgs &a, hipStream_t s) {
  if (a.f32) return run_act_grad<float, float>(a, s);
  return a.dy_f32 ? run_act_grad<float, bf16_t>(a, s) : run_act_grad<bf16_t, bf16_t>(a, s);
}

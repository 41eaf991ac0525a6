// RMS norms before and after a block, fused with the block's gate and the
// residual scales, and their gradients.
//
//   after a block   q = (mean y^2 + eps)^-1/2,  o = alpha h + beta a w y q
//   before a block  r = (mean o^2 + eps)^-1/2,  x = w' o r   (of the unrounded o)
//
// (a: a gate per channel, per token, or none). Every row is read once and
// written once: a row's elements stay in the registers of the threads that
// own its columns between the row sum and the use of its result. All sums are
// fp32. The gradients of the parameters are sums over the rows: a thread adds
// its columns over the rows its workgroup takes, in registers, and a second
// kernel adds the workgroups' partial sums in a fixed order.
#include "norm.h"
#include "vec8.h"

namespace {

constexpr int kCUs = 256;
// bytes of rows that a gradient launch keeps under way on each CU
constexpr int kBwdBytes = 48 * 1024;
// rows from which a workgroup after a block takes two: still several for every CU (measured at 32768 rows of 2560)
constexpr int kTwoRows = 8192;
constexpr int kMaxNarrow = 8192;  // widest row whose elements stay in registers: 1024 threads of 8

// How rows lie on threads: `tr` threads own a row, 8 elements each (a power
// of two below a wave for narrow rows, else whole waves), `rpb` rows per
// workgroup.
struct Map {
  int tr, rpb, threads;
};

Map row_map(int d) {
  const int v = (d + 7) / 8;
  Map m;
  if (v > kMaxNarrow / 8) {
    m.tr = 1024;
  } else if (v > 32) {
    m.tr = (v + 63) / 64 * 64;
  } else {
    m.tr = 8;
    while (m.tr < v) m.tr *= 2;
  }
  m.rpb = m.tr <= 64 ? 256 / m.tr : 1;
  m.threads = m.tr * m.rpb;
  return m;
}

// Workgroups of a gradient launch: each takes rows until none are left and
// writes one partial sum per column. `elem`: bytes of a row's inputs per
// column. Each workgroup has one step's rows under way while it works on the
// step before. As many of them as have 48 KiB under way on a CU measured
// best: at 32768 rows of 2560 (o, dh_in fp32; dx, y bf16: 30 KiB a row) one per
// CU takes 272 us and two 294; at 1024 columns in bf16 (6 KiB a row) eight take
// 58 us, five 65, ten 60 and sixteen 66. More of them only read from more
// places at once, and leave more partial sums.
unsigned bwd_grid(long long rows, const Map &m, int elem) {
  const long long want = (rows + m.rpb - 1) / m.rpb;
  long long per_cu = kBwdBytes / (m.threads * 8 * elem), most = 2048 / m.threads;
  if (per_cu > most) per_cu = most;
  if (per_cu < 1) per_cu = 1;
  return (unsigned)(want < kCUs * per_cu ? want : kCUs * per_cu);
}

// elements between partial sums: whole cache lines
__host__ __device__ __forceinline__ int part_ld(int d) { return (d + 31) / 32 * 32; }

// v plus the value `CTRL` of the DPP controls brings from another lane
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// The sum over `width` lanes (8, 16, 32 or 64), in all of them, without the
// LDS: within a quad by permutation, then each half of 8 and of 16 lanes from
// the other by mirroring (its lanes hold the same sum), then by swapping rows
// of 16 and halves of 32. Through the LDS crossbar the six sums of a gradient
// row cost 36 passes per wave.
__device__ __forceinline__ float wave_sum(float v, int width) {
  v = add_dpp<0xB1>(v);   // quad_perm [1,0,3,2]
  v = add_dpp<0x4E>(v);   // quad_perm [2,3,0,1]
  v = add_dpp<0x141>(v);  // row_half_mirror
  if (width >= 16) v = add_dpp<0x140>(v);  // row_mirror
  if (width >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (width >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Sums of NS values over the tr threads of a row, the result in every one of
// them. Waves of one row add through `red`; its two halves take turns, so one
// barrier per sum is enough: a half is written again only after the barrier
// of the sum between, which every reader of the half has then passed.
template <int NS>
__device__ __forceinline__ void row_sum(float (&s)[NS], int tr, float (*red)[16][NS], int &turn) {
#pragma unroll
  for (int k = 0; k < NS; ++k) s[k] = wave_sum(s[k], tr < 64 ? tr : 64);
  if (tr <= 64) return;
  const int wave = threadIdx.x >> 6, nw = tr >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < NS; ++k) red[turn][wave][k] = s[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NS; ++k) s[k] = 0.f;
#pragma unroll 2  // unrolled further, the loads of all waves' sums would hold a hundred registers
  for (int w = 0; w < nw; ++w) {
#pragma unroll
    for (int k = 0; k < NS; ++k) s[k] += red[turn][w][k];
  }
  turn ^= 1;
}

// A row's sums of squares and of products are formed as if of elements times A.shrink = 2^-k, with 4^k >= d, so that a
// sum is no larger than the largest of its terms and leaves fp32 only where a term itself would (the squares of d
// elements of 1e18 pass 3.4e38 from d = 340 on). A thread's own eight terms are added first and then shrunk: one or two
// products per sum, where shrinking each element took 1% more time in all (32768x2560 bf16). A power of two costs the
// sums no bits; what it moves below fp32 is nothing beside eps, which is 1e-30 at least. The launch passes the powers:
// as arguments they take scalar registers, computed by the threads they took three to six vector registers.
NormArgs scaled(NormArgs a) {
  int k = 0;
  while (1LL << 2 * k < a.d) ++k;
  a.shrink = ldexpf(1.f, -k);
  a.grow = ldexpf(1.f, k);
  a.mean = ldexpf((float)a.d, -2 * k);
  return a;
}

// r of a row from its sum of shrunk squares
__device__ __forceinline__ float row_rms(float sumsq, const NormArgs &A) { return rsqrtf(sumsq / A.mean + A.eps); }

template <typename T>
__device__ __forceinline__ const T *row_of(const void *p, long long row, int d) {
  return reinterpret_cast<const T *>(p) + row * d;
}
template <typename T>
__device__ __forceinline__ T *row_of(void *p, long long row, int d) {
  return reinterpret_cast<T *>(p) + row * d;
}

// The eight columns of a thread: from 8 * c on, or, where the row ends sooner
// (R: its width is no multiple of 8), its last eight. Such a thread computes
// and writes its neighbour's columns a second time, to the same values, and
// leaves them out of its row sums; every element of a row is read before any
// is written (the row sums lie between), so outputs may lie on inputs all the
// same. Threads past the row's end have none.
template <bool R>
struct Cols {
  int at, first;  // first column, and which of the eight is the first of its own
  bool mine;
  __device__ __forceinline__ Cols(int c, int d) {
    mine = c * 8 < d;
    at = R && c * 8 + 8 > d ? d - 8 : c * 8;
    first = c * 8 - at;
  }
  __device__ __forceinline__ float own(int j, float v) const { return !R || j >= first ? v : 0.f; }
};

// ---- forward ----
//
// Which product joins a sum unrounded is written out here. Left to the
// compiler it differs from form to form of a kernel, and with it the last bit
// of a row: with the number of rows, say, or without a next norm.
__device__ __forceinline__ float add_square(float s, float v) { return __builtin_fmaf(v, v, s); }
// alpha h + beta a w n
__device__ __forceinline__ float after_block(const NormArgs &A, float h, float a, float w, float n) {
  return __builtin_fmaf(A.alpha, h, A.beta * a * w * n);
}

// One workgroup per ROWS neighbouring rows (ONE: their addresses are the same
// for all its threads), or per rpb narrow rows. Bound by memory: 32768 rows of
// 2560 with an fp32 stream, bf16 y and x (1.007 GB) take 177 us, 5.7 TB/s, where
// a copy of those arrays in the same pattern takes 165 to 170; bf16 rows of
// 1024 before a block 6.1 TB/s. After a block, with its two sums one behind the
// other, two rows at a time share the barriers and have their loads under way
// together (one row 195 us, four 194); before a block one row is enough (88 us
// at 131072 bf16 rows of 1024, two 92). Workgroups that stay and stride over
// the rows take 206 us, and writing past the caches changes nothing.
template <typename H, typename Y, typename X, bool POST, bool NEXT, bool R, bool ONE, bool TOKEN, int ROWS>
__global__ __launch_bounds__(1024) void k_norm_fwd(NormArgs A, int tr, int rpb) {
  __shared__ float red[2][16][ROWS];
  int turn = 0;
  const int d = A.d, sub = ONE ? 0 : threadIdx.x / tr;
  const Cols<R> cols(ONE ? threadIdx.x : threadIdx.x % tr, d);
  const unsigned c = cols.at;
  const long long row0 = group_index() * rpb * ROWS + sub;
  float o[ROWS][8];
  Raw8<H> ro[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) ro[k] = load_raw(row_of<H>(A.h, row0 + k, d) + c, cols.mine && row0 + k < A.rows);
  if (POST) {
    Raw8<Y> ry[ROWS], ra[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const bool on = cols.mine && row0 + k < A.rows;
      ry[k] = load_raw(row_of<Y>(A.y, row0 + k, d) + c, on);
      if (TOKEN) ra[k] = load_raw(row_of<Y>(A.gate, row0 + k, d) + c, on);
    }
    float y[8], w[8], t[8];
    if (!TOKEN) load_param(A.gate, A.p_f32, c, cols.mine, t);
    load_param(A.w, A.p_f32, c, cols.mine, w);
    float s[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      expand(ry[k], y);
      s[k] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s[k] = add_square(s[k], cols.own(j, y[j]));
      s[k] *= A.shrink * A.shrink;
    }
    row_sum<ROWS>(s, tr, red, turn);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const float q = row_rms(s[k], A);
      expand(ro[k], o[k]);
      expand(ry[k], y);
      if (TOKEN) expand(ra[k], t);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[k][j] = after_block(A, o[k][j], t[j], w[j], y[j] * q);
      store_w(row_of<H>(A.o, row0 + k, d) + c, cols.mine && row0 + k < A.rows, o[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) expand(ro[k], o[k]);
  }
  if (NEXT) {
    float wn[8];
    load_param(A.w_next, A.p_f32, c, cols.mine, wn);
    float s[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      s[k] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s[k] = add_square(s[k], cols.own(j, o[k][j]));
      s[k] *= A.shrink * A.shrink;
    }
    row_sum<ROWS>(s, tr, red, turn);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const float r = row_rms(s[k], A);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[k][j] = wn[j] * (o[k][j] * r);
      store_w(row_of<X>(A.x, row0 + k, d) + c, cols.mine && row0 + k < A.rows, o[k]);
    }
  }
  end_of_stores();
}

// Rows too wide for registers: the row is read again for each step (from the
// caches), one workgroup per row. Each element is written by the thread that
// last reads it, so an output may lie on its input here too.
template <typename H, typename Y, typename X, bool POST, bool NEXT, int W>
__global__ __launch_bounds__(1024) void k_norm_fwd_wide(NormArgs A) {
  __shared__ float red[2][16][1];
  int turn = 0;
  const int d = A.d, v = d / W;
  const long long row = group_index();
  if (row >= A.rows) return;
  const H *h = row_of<H>(A.h, row, d);
  const Y *y = row_of<Y>(A.y, row, d);
  const Y *ta = row_of<Y>(A.gate, row, d);
  float q = 0.f, r = 0.f;
  auto after = [&](int c, float (&o)[W]) {  // o of W columns
    load_w(h + c * W, true, o);
    if (POST) {
      float yy[W], w[W], a[W];
      load_w(y + c * W, true, yy);
      load_param(A.w, A.p_f32, c * W, true, w);
      if (A.token_gate)
        load_w(ta + c * W, true, a);
      else
        load_param(A.gate, A.p_f32, c * W, true, a);
#pragma unroll
      for (int j = 0; j < W; ++j) o[j] = after_block(A, o[j], a[j], w[j], yy[j] * q);
    }
  };
  if (POST) {
    float s[1] = {0.f};
    for (int c = threadIdx.x; c < v; c += 1024) {
      float yy[W];
      load_w(y + c * W, true, yy);
#pragma unroll
      for (int j = 0; j < W; ++j) s[0] = add_square(s[0], yy[j] * A.shrink);
    }
    row_sum<1>(s, 1024, red, turn);
    q = row_rms(s[0], A);
  }
  if (NEXT) {
    float s[1] = {0.f};
    for (int c = threadIdx.x; c < v; c += 1024) {
      float o[W];
      after(c, o);
#pragma unroll
      for (int j = 0; j < W; ++j) s[0] = add_square(s[0], o[j] * A.shrink);
    }
    row_sum<1>(s, 1024, red, turn);
    r = row_rms(s[0], A);
  }
  for (int c = threadIdx.x; c < v; c += 1024) {
    float o[W];
    after(c, o);
    if (POST) store_w(row_of<H>(A.o, row, d) + c * W, true, o);
    if (NEXT) {
      float wn[W];
      load_param(A.w_next, A.p_f32, c * W, true, wn);
#pragma unroll
      for (int j = 0; j < W; ++j) o[j] = wn[j] * (o[j] * r);
      store_w(row_of<X>(A.x, row, d) + c * W, true, o);
    }
  }
}

// ---- gradients ----
//
//   do = dh_in + r (g - (o r) m),  g = dx w',  m = mean(g o r)
//   p  = beta a w do,  dy = q (p - (y q) mean(p y q)),  dh = alpha do
//   over the rows: dw' = sum dx o r;  S = sum do a_t y q (a_t: the gate per
//   token, or 1), from which dw = beta a_c S and, per channel, da = beta w S;
//   per token da = beta do w y q.
//
// mean(p y q) needs do, which needs r and m. Put in, sum(p y) is a sum of
// three products that do not: with k = beta a w,
//   sum(k do y) = sum(k dh_in y) + r sum(k g y) - r m (r sum(k o y)),
// so one pass over the registers and one exchange between the waves gives all
// the row's sums. r and m meet o and y as n = o r and y q only: r^2 by itself
// would lose its bits below 1e-38, where o is large.

// What a gradient call keeps of one row after its sums.
struct RowStat {
  float r, rm, q, qs;  // m = mean(g n), s = mean(p y q)
};

template <bool POST, bool NEXT>
__device__ __forceinline__ RowStat row_stat(const float (&s)[6], const NormArgs &A) {
  RowStat t{0.f, 0.f, 0.f, 0.f};
  const float inv = 1.f / (float)A.d;
  float py = s[3];  // shrunk
  if (NEXT) {
    t.r = row_rms(s[0], A);
    const float grown = t.r * A.grow;
    t.rm = t.r * (s[1] * grown * inv);
    py += t.r * s[4] - t.rm * (grown * s[5]);
  }
  if (POST) {
    t.q = row_rms(s[2], A);
    t.qs = t.q * (py * (t.q * A.grow) * inv);
  }
  return t;
}

// the terms of one element of the row's sums
template <bool POST, bool NEXT>
__device__ __forceinline__ void add_terms(float (&s)[6], float o, float g, float di, float y, float k) {
  if (NEXT) {
    s[0] += o * o;
    s[1] += g * o;
  }
  if (POST) {
    const float ky = k * y;
    s[2] += y * y;
    s[3] += ky * di;
    if (NEXT) {
      s[4] += ky * g;
      s[5] += ky * o;
    }
  }
}

// A row's inputs, as they lie in memory.
template <typename H, typename Y, typename X, bool POST, bool NEXT, bool TOKEN>
struct BwdRow {
  Raw8<H> o, di;
  Raw8<X> dx;
  Raw8<Y> y, a;
  __device__ __forceinline__ void load(const NormArgs &A, long long row, unsigned c, bool on) {
    const int d = A.d;
    if (NEXT) {
      o = load_raw(row_of<H>(A.h, row, d) + c, on);
      dx = load_raw(row_of<X>(A.dx, row, d) + c, on);
    }
    di = load_raw(row_of<H>(A.dh_in, row, d) + c, on && A.dh_in);
    if (POST) y = load_raw(row_of<Y>(A.y, row, d) + c, on);
    if (POST && TOKEN) a = load_raw(row_of<Y>(A.gate, row, d) + c, on);
  }
};

// Partial sums of workgroup b, [b][2][part_ld(d)]: the gradient of w', then S.
// Bound by memory: 32768 rows of 2560 as above (1.51 GB) take 269 us with the
// sums over the workgroups, 5.6 TB/s (up to a fifth more in the first 20 ms of a
// load); 32768 bf16 rows of 1024 (0.27 GB) 57 us.
// The loads of a workgroup's next row are issued before this row's results are
// stored: waits for memory operations are counted in their order, so loads
// behind the stores would be waited for together with them. AHEAD: not where
// a thread of 1024, with 128 registers, would have to spill for it (13 to 75 of
// them): 8192 rows of 5120 with an fp32 stream take 156 us so against 174, with
// a gate per token 184 against 409. bf16 rows without that gate spill none and
// gain from it (119 us without, 111 with), as a first norm's do (125, 120).
template <typename H, typename Y, typename X, bool POST, bool NEXT, bool R, bool ONE, bool TOKEN, int MOST>
__global__ __launch_bounds__(MOST) void k_norm_bwd(NormArgs A, int tr, int rpb) {
  __shared__ float red[2][16][6];
  __shared__ float acc[2][ONE ? 1 : 256 * 8];  // workgroups of several rows (256 threads) add their rows' columns here
  int turn = 0;
  const int d = A.d, sub = ONE ? 0 : threadIdx.x / tr;
  const Cols<R> cols(ONE ? threadIdx.x : threadIdx.x % tr, d);
  const unsigned c = cols.at;
  const bool mine = cols.mine;
  float w[8], wn[8], k[8], dwn[8], ds[8];
  if (POST) {
    load_param(A.w, A.p_f32, c, mine, w);
    load_param(TOKEN ? nullptr : A.gate, A.p_f32, c, mine, k);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] *= A.beta;
      k[j] *= w[j];
    }
  }
  if (NEXT) load_param(A.w_next, A.p_f32, c, mine, wn);
#pragma unroll
  for (int j = 0; j < 8; ++j) dwn[j] = ds[j] = 0.f;

  const long long step = (long long)gridDim.x * rpb;
  long long row = (long long)blockIdx.x * rpb + sub;
  BwdRow<H, Y, X, POST, NEXT, TOKEN> in;
  constexpr bool AHEAD = MOST <= 512 || !POST || !NEXT || (!TOKEN && sizeof(H) == 2);
  if (AHEAD) in.load(A, row, c, mine && row < A.rows);
  for (long long row0 = (long long)blockIdx.x * rpb; row0 < A.rows; row0 += step, row += step) {
    const bool on = mine && row < A.rows;
    float o[8], g[8], di[8], y[8], a[8];
    if (!AHEAD) in.load(A, row, c, on);
    if (NEXT) {
      expand(in.o, o);
      expand(in.dx, g);
    }
    expand(in.di, di);
    if (POST) expand(in.y, y);
    if (POST && TOKEN) expand(in.a, a);
    if (AHEAD) in.load(A, row + step, c, mine && row + step < A.rows);
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      add_terms<POST, NEXT>(s, NEXT ? cols.own(j, o[j]) : 0.f, NEXT ? g[j] * wn[j] : 0.f, di[j],
                            POST ? cols.own(j, y[j]) : 0.f, !POST ? 0.f : TOKEN ? k[j] * a[j] : k[j]);
    if (NEXT) {
      s[0] *= A.shrink * A.shrink;
      s[1] *= A.shrink;
    }
    if (POST) {
      s[2] *= A.shrink * A.shrink;
      s[3] *= A.shrink;
    }
    if (POST && NEXT) {
      s[4] *= A.shrink;
      s[5] *= A.shrink * A.shrink;
    }
    row_sum<6>(s, tr, red, turn);
    const RowStat t = row_stat<POST, NEXT>(s, A);
    float dh[8], dy[8], da[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = di[j];
      if (NEXT) {
        const float n = o[j] * t.r;
        v += t.r * (g[j] * wn[j]) - t.rm * n;
        dwn[j] += g[j] * n;
      }
      dh[j] = A.alpha * v;
      if (POST) {
        const float yn = y[j] * t.q, ta = TOKEN ? a[j] : 1.f;
        ds[j] += v * ta * yn;
        da[j] = v * w[j] * yn;
        dy[j] = t.q * (k[j] * ta * v) - t.qs * yn;
      }
    }
    store_w(row_of<H>(A.dh, row, d) + c, on, dh);
    if (POST) {
      store_w(row_of<Y>(A.dy, row, d) + c, on, dy);
      if (TOKEN) store_w(row_of<Y>(A.dgate_t, row, d) + c, on, da);
    }
  }
  if (!A.part) return;
  const int ld = part_ld(d);
  float *part = A.part + (long long)blockIdx.x * 2 * ld;
  if (ONE) {
    if (NEXT) store_w(part + c, mine, dwn);
    if (POST) store_w(part + ld + c, mine, ds);
    return;
  }
  if (mine) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[0][ONE ? 0 : sub * tr * 8 + c + j] = dwn[j];
      acc[1][ONE ? 0 : sub * tr * 8 + c + j] = ds[j];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < d; i += blockDim.x) {
    float s0 = 0.f, s1 = 0.f;
    for (int u = 0; u < rpb; ++u) {
      s0 += acc[0][ONE ? 0 : u * tr * 8 + i];
      s1 += acc[1][ONE ? 0 : u * tr * 8 + i];
    }
    if (NEXT) part[i] = s0;
    if (POST) part[ld + i] = s1;
  }
}

// Rows too wide for registers: sums in one pass over the row, results in a
// second, and the columns' partial sums in the workgroup's slice of the
// workspace (each element only ever touched by the same thread).
template <typename H, typename Y, typename X, bool POST, bool NEXT, int W>
__global__ __launch_bounds__(1024) void k_norm_bwd_wide(NormArgs A) {
  __shared__ float red[2][16][6];
  int turn = 0;
  const int d = A.d, v = d / W;
  const int ld = part_ld(d);
  float *part = A.part ? A.part + (long long)blockIdx.x * 2 * ld : nullptr;
  bool first = true;
  for (long long row = blockIdx.x; row < A.rows; row += gridDim.x) {
    float o[W], g[W], di[W], y[W], a[W], w[W], k[W], dxv[W];
    auto read = [&](int c) {
      if (NEXT) {
        load_w(row_of<H>(A.h, row, d) + c * W, true, o);
        load_w(row_of<X>(A.dx, row, d) + c * W, true, dxv);
        load_param(A.w_next, A.p_f32, c * W, true, g);
#pragma unroll
        for (int j = 0; j < W; ++j) g[j] *= dxv[j];
      }
      load_w(row_of<H>(A.dh_in, row, d) + c * W, A.dh_in != nullptr, di);
      if (POST) {
        load_w(row_of<Y>(A.y, row, d) + c * W, true, y);
        load_param(A.w, A.p_f32, c * W, true, w);
        if (A.token_gate) {
          load_w(row_of<Y>(A.gate, row, d) + c * W, true, a);
#pragma unroll
          for (int j = 0; j < W; ++j) k[j] = 1.f;
        } else {
          load_param(A.gate, A.p_f32, c * W, true, k);
#pragma unroll
          for (int j = 0; j < W; ++j) a[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          w[j] *= A.beta;
          k[j] *= w[j] * a[j];
        }
      }
    };
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c = threadIdx.x; c < v; c += 1024) {
      read(c);
#pragma unroll
      for (int j = 0; j < W; ++j)
        add_terms<POST, NEXT>(s, NEXT ? o[j] * A.shrink : 0.f, NEXT ? g[j] : 0.f, di[j], POST ? y[j] * A.shrink : 0.f,
                              POST ? k[j] : 0.f);
    }
    row_sum<6>(s, 1024, red, turn);
    const RowStat t = row_stat<POST, NEXT>(s, A);
    for (int c = threadIdx.x; c < v; c += 1024) {
      read(c);
      float dh[W], dy[W], da[W], dwn[W], ds[W];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float u = di[j];
        if (NEXT) {
          const float n = o[j] * t.r;
          u += t.r * g[j] - t.rm * n;
          dwn[j] = dxv[j] * n;
        }
        dh[j] = A.alpha * u;
        if (POST) {
          const float yn = y[j] * t.q;
          ds[j] = u * a[j] * yn;
          da[j] = u * w[j] * yn;
          dy[j] = t.q * (k[j] * u) - t.qs * yn;
        }
      }
      store_w(row_of<H>(A.dh, row, d) + c * W, true, dh);
      if (POST) {
        store_w(row_of<Y>(A.dy, row, d) + c * W, true, dy);
        if (A.token_gate) store_w(row_of<Y>(A.dgate_t, row, d) + c * W, true, da);
      }
      if (part) {
        float old[W];
        if (NEXT) {
          load_w(part + c * W, !first, old);
#pragma unroll
          for (int j = 0; j < W; ++j) old[j] += dwn[j];
          store_w(part + c * W, true, old);
        }
        if (POST) {
          load_w(part + ld + c * W, !first, old);
#pragma unroll
          for (int j = 0; j < W; ++j) old[j] += ds[j];
          store_w(part + ld + c * W, true, old);
        }
      }
    }
    first = false;
  }
}

// The parameters' gradients from the workgroups' partial sums (nparts of
// them; none for a call without rows). A workgroup takes 32 columns, a cache
// line of each partial sum: 8 threads across it, 128 down the partial sums.
constexpr int kDown = 128;
__global__ __launch_bounds__(kDown * 8) void k_norm_params(NormArgs A, int nparts) {
  __shared__ f32x4 sum[kDown][8];
  const int d = A.d, which = blockIdx.y, ld = part_ld(d);
  if (which == 0 ? !A.dw_next : (!A.dw && !A.dgate_c)) return;
  const int across = threadIdx.x & 7, down = threadIdx.x >> 3;
  const float *p = A.part + (long long)which * ld + blockIdx.x * 32 + across * 4;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int b = down; b < nparts; b += kDown) s += *reinterpret_cast<const f32x4 *>(p + (long long)b * 2 * ld);
  sum[down][across] = s;
  for (int half = kDown / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (down < half) sum[down][across] += sum[down + half][across];
  }
  __syncthreads();
  const int i = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x >= 32 || i >= d) return;
  const float t = sum[0][threadIdx.x / 4][threadIdx.x % 4];
  if (which == 0) {
    A.dw_next[i] = t;
    return;
  }
  auto param = [&](const void *q) {
    if (!q) return 1.f;
    return A.p_f32 ? reinterpret_cast<const float *>(q)[i] : bf16_to_f32(reinterpret_cast<const bf16_t *>(q)[i]);
  };
  if (A.dw) A.dw[i] = A.beta * (A.token_gate ? 1.f : param(A.gate)) * t;
  if (A.dgate_c) A.dgate_c[i] = A.beta * param(A.w) * t;
}

// ---- which instance ----
template <typename H, typename Y, typename X, bool POST, bool NEXT, bool R, bool ONE, int ROWS>
void fwd_rows(const NormArgs &a, const Map &m, hipStream_t s) {
  const dim3 grid = group_grid((a.rows + m.rpb * ROWS - 1) / (m.rpb * ROWS)), block(m.threads);
  if (POST && a.token_gate)
    hipLaunchKernelGGL((k_norm_fwd<H, Y, X, POST, NEXT, R, ONE, POST, ROWS>), grid, block, 0, s, a, m.tr, m.rpb);
  else
    hipLaunchKernelGGL((k_norm_fwd<H, Y, X, POST, NEXT, R, ONE, false, ROWS>), grid, block, 0, s, a, m.tr, m.rpb);
}

template <typename H, typename Y, typename X, bool POST, bool NEXT, bool R, bool ONE>
void fwd_form(const NormArgs &a, const Map &m, hipStream_t s) {
  if (ONE && POST && a.rows >= kTwoRows)
    fwd_rows<H, Y, X, POST, NEXT, R, ONE, ONE && POST ? 2 : 1>(a, m, s);
  else
    fwd_rows<H, Y, X, POST, NEXT, R, ONE, 1>(a, m, s);
}

template <typename H, typename Y, typename X, bool POST, bool NEXT>
hipError_t fwd(const NormArgs &a, hipStream_t s) {
  const Map m = row_map(a.d);
  const dim3 grid = group_grid(a.rows);
  if (a.d > kMaxNarrow && a.d % 8)
    hipLaunchKernelGGL((k_norm_fwd_wide<H, Y, X, POST, NEXT, 1>), grid, dim3(1024), 0, s, a);
  else if (a.d > kMaxNarrow)
    hipLaunchKernelGGL((k_norm_fwd_wide<H, Y, X, POST, NEXT, 8>), grid, dim3(1024), 0, s, a);
  else if (m.rpb == 1)
    a.d % 8 ? fwd_form<H, Y, X, POST, NEXT, true, true>(a, m, s) : fwd_form<H, Y, X, POST, NEXT, false, true>(a, m, s);
  else
    a.d % 8 ? fwd_form<H, Y, X, POST, NEXT, true, false>(a, m, s)
            : fwd_form<H, Y, X, POST, NEXT, false, false>(a, m, s);
  return hipGetLastError();
}

template <typename H, typename Y, typename X, bool POST, bool NEXT, bool R, bool ONE, bool TOKEN>
void bwd_launch(const NormArgs &a, const Map &m, unsigned grid, hipStream_t s) {
  // up to 512 threads a kernel may hold 256 registers each and spills none (340 us and more at 32768 rows of 2560 with
  // the 128 that 1024 threads allow, where it loads ahead)
  if (!ONE || m.threads <= 512)
    hipLaunchKernelGGL((k_norm_bwd<H, Y, X, POST, NEXT, R, ONE, TOKEN, 512>), dim3(grid), dim3(m.threads), 0, s, a,
                       m.tr, m.rpb);
  else
    hipLaunchKernelGGL((k_norm_bwd<H, Y, X, POST, NEXT, R, ONE, TOKEN, ONE ? 1024 : 512>), dim3(grid),
                       dim3(m.threads), 0, s, a, m.tr, m.rpb);
}

template <typename H, typename Y, typename X, bool POST, bool NEXT, bool R, bool ONE>
void bwd_form(const NormArgs &a, const Map &m, unsigned grid, hipStream_t s) {
  if (POST && a.token_gate)
    bwd_launch<H, Y, X, POST, NEXT, R, ONE, POST>(a, m, grid, s);
  else
    bwd_launch<H, Y, X, POST, NEXT, R, ONE, false>(a, m, grid, s);
}

template <typename H, typename Y, typename X, bool POST, bool NEXT>
hipError_t bwd(const NormArgs &a, hipStream_t s) {
  const Map m = row_map(a.d);
  constexpr int elem = (NEXT ? sizeof(H) + sizeof(X) : 0) + sizeof(H) + (POST ? sizeof(Y) : 0);
  const unsigned grid = bwd_grid(a.rows, m, elem);
  if (grid > 0) {
    if (a.d > kMaxNarrow && a.d % 8)
      hipLaunchKernelGGL((k_norm_bwd_wide<H, Y, X, POST, NEXT, 1>), dim3(grid), dim3(1024), 0, s, a);
    else if (a.d > kMaxNarrow)
      hipLaunchKernelGGL((k_norm_bwd_wide<H, Y, X, POST, NEXT, 8>), dim3(grid), dim3(1024), 0, s, a);
    else if (m.rpb == 1)
      a.d % 8 ? bwd_form<H, Y, X, POST, NEXT, true, true>(a, m, grid, s)
              : bwd_form<H, Y, X, POST, NEXT, false, true>(a, m, grid, s);
    else
      a.d % 8 ? bwd_form<H, Y, X, POST, NEXT, true, false>(a, m, grid, s)
              : bwd_form<H, Y, X, POST, NEXT, false, false>(a, m, grid, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.part) hipLaunchKernelGGL(k_norm_params, dim3((a.d + 31) / 32, 2), dim3(kDown * 8), 0, s, a, (int)grid);
  return hipGetLastError();
}

}  // namespace

size_t norm_ws_bytes(long long rows, int d) {
  const unsigned grid = bwd_grid(rows, row_map(d), 4);  // the least of any types
  return (size_t)(grid > 0 ? grid : 1) * 2 * part_ld(d) * sizeof(float);
}

#define NORM_CASES(CALL)                                                                                  \
  if (post && next) {                                                                                     \
    if (t.h && t.y && t.x) return CALL<float, float, float, true, true>(a, s);                            \
    if (t.h && t.y) return CALL<float, float, bf16_t, true, true>(a, s);                                  \
    if (t.h && !t.y && !t.x) return CALL<float, bf16_t, bf16_t, true, true>(a, s);                        \
    if (!t.h && !t.y && !t.x) return CALL<bf16_t, bf16_t, bf16_t, true, true>(a, s);                      \
  } else if (post) {                                                                                      \
    if (t.h && t.y) return CALL<float, float, float, true, false>(a, s);                                  \
    if (t.h) return CALL<float, bf16_t, bf16_t, true, false>(a, s);                                       \
    if (!t.y) return CALL<bf16_t, bf16_t, bf16_t, true, false>(a, s);                                     \
  } else {                                                                                                \
    if (t.h && t.x) return CALL<float, float, float, false, true>(a, s);                                  \
    if (t.h) return CALL<float, float, bf16_t, false, true>(a, s);                                        \
    if (!t.x) return CALL<bf16_t, bf16_t, bf16_t, false, true>(a, s);                                     \
  }                                                                                                       \
  return hipErrorInvalidValue

hipError_t launch_norm_fwd(const NormArgs &args, NormTypes t, hipStream_t s) {
  if (args.rows <= 0) return hipSuccess;
  const NormArgs a = scaled(args);
  const bool post = a.y != nullptr, next = a.x != nullptr;
  NORM_CASES(fwd);
}

hipError_t launch_norm_bwd(const NormArgs &args, NormTypes t, bool post, bool next, hipStream_t s) {
  const NormArgs a = scaled(args);
  NORM_CASES(bwd);
}

// Token embedding with a scale, x[t] = scale * E[ids[t]], and its gradient,
// dE[v] = scale * sum of dx[t] over the tokens t with ids[t] = v. An id outside
// [0, vocab) gives a zero row and takes no gradient (the zero target rows of
// the layer follow the same reading).
//
// The gradient does not add with atomics, whose order would change its bits:
// the tokens are sorted by id, stably, so that each table row's tokens lie
// together in the order of their positions, and each row is summed in fp32 by
// one wave in that order. Ids are skewed in real text, so a row of more than
// kChunk tokens is cut at multiples of kChunk sorted tokens; the pieces are
// summed side by side and joined in order. The sort is a radix sort of (id,
// position) by counting: per pass, each workgroup counts its tile's digits,
// and then places its tokens from the counts of all tiles.
#include "embed.h"
#include "vec8.h"

namespace {

// x larger than this is written past the caches: the last level of them holds 256 MiB, and at half a GiB little of it
// would be left for the next kernel
constexpr double kStreamBytes = 512.0 * (1 << 20);
constexpr int kMaxTiles = 256;   // of a sort: a workgroup reads the counts of all of them
constexpr int kMinTile = 1024;   // tokens
constexpr int kMaxDigit = 9;     // bits
constexpr int kSortThreads = 256, kSortWaves = kSortThreads / 64;
constexpr long long kMaxGroups = 1 << 22;  // of a launch: threads of a grid are counted in 32 bits
constexpr int kClearPerGroup = 2048;  // table rows whose segments one workgroup clears
constexpr int kChunk = 64;       // sorted tokens of one piece of a long row

// ---- lookup ----

// A workgroup takes one row (ONE: its id is the same for all threads and its
// addresses need no vector arithmetic), or, of narrow rows, `rpb` rows of `tr`
// threads. There is a workgroup for every row: a grid that keeps the card
// full and strides over the rows measured 470 us on 131072 bf16 rows of 2560
// into fp32 where this one takes 290 (1.52 GB: 5.3 TB/s), since rows that run
// at the same time then lie side by side in memory. STREAM: x is too large to
// be found in the caches later; its rows are written past them (362 us without;
// at 168 MB 60 us with it and 42 without).
template <typename E, typename X, bool R, bool ONE, bool STREAM>
__global__ __launch_bounds__(1024) void k_embed(EmbedArgs A, int tr, int rpb) {
  const int sub = ONE ? 0 : threadIdx.x / tr, d = A.d;
  const long long row = group_index() * rpb + sub;
  if (row >= A.ids.n) return;
  const int id = A.ids.at((unsigned)row);
  const bool on = id >= 0 && id < A.vocab;
  const E *src = reinterpret_cast<const E *>(A.E) + (long long)(on ? id : 0) * d;
  X *dst = reinterpret_cast<X *>(A.x) + row * d;
  for (int c8 = ONE ? threadIdx.x : threadIdx.x % tr; c8 * 8 < d; c8 += tr) {
    // the last columns of a ragged row: its last eight, some of which the neighbour writes too, to the same values
    const int c = R && c8 * 8 + 8 > d ? d - 8 : c8 * 8;
    float v[8];
    load_w(src + c, on, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= A.scale;
    if (STREAM)
      stream_w(dst + c, true, v);
    else
      store_w(dst + c, true, v);
  }
}

// ---- sort ----

// What a sort of n tokens with keys 0 .. vocab (vocab: no row) looks like.
struct SortPlan {
  int tile, tiles, passes, digit;  // tokens per tile, tiles, passes, bits of a digit
};

SortPlan sort_plan(long long n, int vocab) {
  SortPlan p;
  long long tile = (n + kMaxTiles - 1) / kMaxTiles;
  tile = (tile + kMinTile - 1) / kMinTile * kMinTile;
  if (tile < kMinTile) tile = kMinTile;
  p.tile = (int)tile;
  p.tiles = (int)((n + tile - 1) / tile);
  int bits = 1;
  while (((long long)vocab >> bits) != 0) ++bits;
  p.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  p.digit = (bits + p.passes - 1) / p.passes;
  return p;
}

struct Run {
  int start, end;  // sorted tokens of a table row; 0, 0: none
};

struct SortArgs {
  TokenIds ids;
  int vocab, shift, bins, tile, tiles;
  const uint32_t *key_in, *pos_in;  // NULL in the first pass: the ids themselves
  uint32_t *key_out, *pos_out;
  uint32_t *hist;  // [tiles][bins]
  Run *seg;        // [vocab], cleared by the first pass's counts
  __device__ __forceinline__ uint32_t key(int i) const {
    if (key_in) return key_in[i];
    const int id = ids.at((unsigned)i);
    return id >= 0 && id < vocab ? (uint32_t)id : (uint32_t)vocab;
  }
};

// hist[tile][digit]: how often each digit occurs in the tile
__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs S) {
  __shared__ uint32_t cnt[1 << kMaxDigit];
  for (int i = threadIdx.x; i < S.bins; i += kSortThreads) cnt[i] = 0;
  if (!S.key_in) {
    for (long long v = (long long)blockIdx.x * kSortThreads + threadIdx.x; v < S.vocab;
         v += (long long)gridDim.x * kSortThreads)
      S.seg[v] = Run{0, 0};
  }
  if ((int)blockIdx.x >= S.tiles) return;  // here to clear only
  __syncthreads();
  const long long t0 = (long long)blockIdx.x * S.tile;
  const int hi = (int)(t0 + S.tile < S.ids.n ? t0 + S.tile : S.ids.n);
  for (int i = (int)t0 + threadIdx.x; i < hi; i += kSortThreads)
    atomicAdd(&cnt[(S.key(i) >> S.shift) & (S.bins - 1)], 1u);
  __syncthreads();
  for (int i = threadIdx.x; i < S.bins; i += kSortThreads) S.hist[(long long)blockIdx.x * S.bins + i] = cnt[i];
}

// Places the tile's tokens: behind all tokens of a smaller digit, and those of
// the same digit in earlier tiles, earlier waves' parts of the tile (each wave
// owns a run of it) and earlier steps of the wave.
__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortArgs S) {
  __shared__ uint32_t next[kSortWaves][1 << kMaxDigit];  // where a wave's next token of a digit goes
  __shared__ uint32_t wsum[kSortWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < kSortWaves * S.bins; i += kSortThreads) next[i / S.bins][i % S.bins] = 0;
  __syncthreads();
  const long long t0 = (long long)blockIdx.x * S.tile;
  const int run = S.tile / kSortWaves;
  const long long w0 = t0 + (long long)wave * run;
  const int lo = (int)(w0 < S.ids.n ? w0 : S.ids.n), hi = (int)(w0 + run < S.ids.n ? w0 + run : S.ids.n);
  for (int i = lo + lane; i < hi; i += 64) atomicAdd(&next[wave][(S.key(i) >> S.shift) & (S.bins - 1)], 1u);
  __syncthreads();
  // two neighbouring digits per thread (at most 512 of them): their totals, and the part before this tile
  uint32_t total[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = threadIdx.x * 2 + k;
    if (b >= S.bins) break;
    for (int t = 0; t < S.tiles; ++t) {
      const uint32_t h = S.hist[(long long)t * S.bins + b];
      total[k] += h;
      before[k] += t < (int)blockIdx.x ? h : 0;
    }
  }
  // exclusive sum of the totals over the digits
  uint32_t inc = total[0] + total[1];
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  uint32_t base = inc - total[0] - total[1];
  for (int w = 0; w < wave; ++w) base += wsum[w];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = threadIdx.x * 2 + k;
    if (b >= S.bins) break;
    uint32_t at = base + before[k];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = next[w][b];
      next[w][b] = at;
      at += c;
    }
    base += total[k];
  }
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += 64) {
    const int i = i0 + lane;
    const bool in = i < hi;
    const uint32_t key = in ? S.key(i) : 0;
    const int dg = (int)((key >> S.shift) & (S.bins - 1));
    // the lanes with the same digit
    uint64_t same = __ballot(in);
    for (int bit = 1; bit < S.bins; bit <<= 1) {
      const uint64_t one = __ballot(in && (dg & bit));
      same &= (dg & bit) ? one : ~one;
    }
    if (in) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int first = __ffsll((unsigned long long)same) - 1;
      uint32_t at = 0;
      if (lane == first) at = atomicAdd(&next[wave][dg], (uint32_t)__popcll(same));
      at = __shfl(at, first) + rank;
      S.key_out[at] = key;
      S.pos_out[at] = S.pos_in ? S.pos_in[i] : (uint32_t)i;
    }
  }
}

// seg[v]: the sorted tokens of table row v
__global__ __launch_bounds__(256) void k_segments(const uint32_t *key, int n, int vocab, Run *seg) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const uint32_t k = key[i];
  if (k >= (uint32_t)vocab) return;
  if (i == 0 || key[i - 1] != k) seg[k].start = (int)i;
  if (i == n - 1 || key[i + 1] != k) seg[k].end = (int)i + 1;
}

// ---- sums ----

struct SumArgs {
  const void *dx;
  void *dE;
  const uint32_t *key, *pos;  // sorted
  const Run *seg;
  float *part;  // [chunks][2][d]
  int n, vocab, d, accumulate;
  float scale;
};

// The scaled sum of eight columns into the table's gradient. `first`: a
// thread at the end of a ragged row owns its columns from there on only.
template <typename G>
__device__ __forceinline__ void put(G *p, int first, int accumulate, float scale, float (&s)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] *= scale;
  if (first) {
    for (int j = 7; j >= 1; --j) {
      float v[1] = {s[j]}, old[1] = {0.f};
      if (j < first) break;
      if (accumulate) load_w(p + j, true, old);
      v[0] += old[0];
      store_w(p + j, true, v);
    }
    return;
  }
  if (accumulate) {
    float old[8];
    load_w(p, true, old);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += old[j];
  }
  store_w(p, true, s);
}

// A table row's tokens, in order, into NV vectors of 8 columns per lane of a
// wave. An item is a table row, or, when the sums are added to dE, a sorted
// token, which counts if it is the first of its row. Rows of more than kChunk
// tokens are left to k_long.
template <typename D, typename G, int NV, bool R>
__device__ __forceinline__ void row_item(const SumArgs &S, long long item, int part) {
  const int lane = threadIdx.x & 63, d = S.d;
  const int c0 = part * (NV * 512) + lane * 8;
  long long v = item;
  if (S.accumulate) {
    v = S.key[item];
    if (v >= S.vocab || (item > 0 && S.key[item - 1] == (uint32_t)v)) return;
  }
  const Run g = S.seg[v];
  if (g.end - g.start > kChunk) return;
  float acc[NV][8];
  int at[NV], first[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = c0 + k * 512;
    at[k] = R && c + 8 > d ? d - 8 : c;
    first[k] = c >= d ? 8 : c - at[k];  // 8: no columns here
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[k][j] = 0.f;
  }
  for (int i = g.start; i < g.end; ++i) {
    const D *row = reinterpret_cast<const D *>(S.dx) + (long long)S.pos[i] * d;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float t[8];
      load_w(row + at[k], first[k] < 8, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[k][j] += t[j];
    }
  }
  G *out = reinterpret_cast<G *>(S.dE) + v * d;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (first[k] < 8) put(out + at[k], R ? first[k] : 0, S.accumulate, S.scale, acc[k]);
}

// one wave per (item, part of the columns)
template <typename D, typename G, int NV, bool R>
__global__ __launch_bounds__(256) void k_rows(SumArgs S, long long items, int parts) {
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  for (long long i = w; i < items * parts; i += (long long)gridDim.x * 4)
    row_item<D, G, NV, R>(S, i / parts, (int)(i % parts));
}

// The long rows with tokens in a chunk: the one the chunk opens with (which may
// have begun earlier), and the one it closes with if that is another. A long
// row cannot lie inside a chunk, so there are no others.
struct ChunkRows {
  int v[2], lo[2], hi[2];  // table row (-1: none) and its sorted tokens in this chunk
  Run seg[2];
  __device__ __forceinline__ ChunkRows(const SumArgs &S, int chunk) {
    const int a = chunk * kChunk, b = a + kChunk < S.n ? a + kChunk : S.n;
    const uint32_t k0 = S.key[a], k1 = S.key[b - 1];
    take(S, 0, k0, a, b);
    v[1] = -1;
    if (k1 != k0) take(S, 1, k1, a, b);
  }
  __device__ __forceinline__ void take(const SumArgs &S, int i, uint32_t k, int a, int b) {
    v[i] = -1;
    if (k >= (uint32_t)S.vocab) return;
    seg[i] = S.seg[k];
    if (seg[i].end - seg[i].start <= kChunk) return;
    v[i] = (int)k;
    lo[i] = seg[i].start > a ? seg[i].start : a;
    hi[i] = seg[i].end < b ? seg[i].end : b;
  }
};

// part[chunk][i]: the sum of a long row's tokens in this chunk
template <typename D, bool R>
__global__ __launch_bounds__(256) void k_long(SumArgs S) {
  const ChunkRows r(S, blockIdx.x);
  const int d = S.d;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 8;
  if (c >= d) return;
  const int at = R && c + 8 > d ? d - 8 : c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (r.v[i] < 0) continue;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int t = r.lo[i]; t < r.hi[i]; ++t) {
      float v[8];
      load_w(reinterpret_cast<const D *>(S.dx) + (long long)S.pos[t] * d + at, true, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[j];
    }
    store_w(S.part + ((long long)blockIdx.x * 2 + i) * d + at, true, acc);
  }
}

// A long row from its pieces: workgroup (chunk, 512 columns) for the long row
// that begins in the chunk, each wave a run of the pieces, the waves' sums
// joined in order.
constexpr int kJoinWaves = 8;
template <typename G, bool R>
__global__ __launch_bounds__(kJoinWaves * 64) void k_join(SumArgs S) {
  __shared__ float sum[kJoinWaves][64][9];
  const ChunkRows r(S, blockIdx.x);
  const int a = blockIdx.x * kChunk, d = S.d;
  int i = -1;
  if (r.v[1] >= 0)
    i = 1;
  else if (r.v[0] >= 0 && r.seg[0].start >= a)
    i = 0;
  if (i < 0) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = (blockIdx.y * 64 + lane) * 8;
  const int at = R && c + 8 > d ? d - 8 : c;
  const int last = (r.seg[i].end - 1) / kChunk;  // pieces: (blockIdx.x, i), then (j, 0) up to the last chunk
  const int pieces = last - (int)blockIdx.x + 1, run = (pieces + kJoinWaves - 1) / kJoinWaves;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < d) {
    const int p0 = wave * run, p1 = p0 + run < pieces ? p0 + run : pieces;
#pragma unroll 8
    for (int p = p0; p < p1; ++p) {
      float v[8];
      load_w(S.part + (((long long)blockIdx.x + p) * 2 + (p == 0 ? i : 0)) * d + at, true, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[wave][lane][j] = acc[j];
  __syncthreads();
  if (wave != 0 || c >= d) return;
  for (int w = 1; w < kJoinWaves; ++w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += sum[w][lane][j];
  }
  put(reinterpret_cast<G *>(S.dE) + (long long)r.v[i] * d + at, R ? c - at : 0, S.accumulate, S.scale, acc);
}

// ---- which instance ----

template <typename E, typename X, bool R, bool ONE>
void embed_form(const EmbedArgs &a, dim3 grid, int tr, int rpb, hipStream_t s) {
  // not ragged rows: parts of cache lines written past the caches cost more (491 MB: 187 us, 129 through them)
  if (!R && (double)a.ids.n * a.d * sizeof(X) > kStreamBytes)
    hipLaunchKernelGGL((k_embed<E, X, R, ONE, !R>), grid, dim3(tr * rpb), 0, s, a, tr, rpb);
  else
    hipLaunchKernelGGL((k_embed<E, X, R, ONE, false>), grid, dim3(tr * rpb), 0, s, a, tr, rpb);
}

template <typename E, typename X>
hipError_t embed(const EmbedArgs &a, hipStream_t s) {
  const int v = (a.d + 7) / 8;
  int tr = 8;
  while (tr < v && tr < 64) tr *= 2;
  if (v > 64) tr = v >= 1024 ? 1024 : (v + 63) / 64 * 64;
  const int rpb = tr <= 64 ? 256 / tr : 1;
  const dim3 grid = group_grid((a.ids.n + rpb - 1LL) / rpb);
  if (rpb > 1)
    a.d % 8 ? embed_form<E, X, true, false>(a, grid, tr, rpb, s) : embed_form<E, X, false, false>(a, grid, tr, rpb, s);
  else
    a.d % 8 ? embed_form<E, X, true, true>(a, grid, tr, rpb, s) : embed_form<E, X, false, true>(a, grid, tr, rpb, s);
  return hipGetLastError();
}

template <typename D, typename G, int NV>
void rows_nv(const SumArgs &S, long long items, int parts, hipStream_t s) {
  const long long groups = (items * parts + 3) / 4;
  const dim3 grid((unsigned)(groups < kMaxGroups ? groups : kMaxGroups));
  if (S.d % 8)
    hipLaunchKernelGGL((k_rows<D, G, NV, true>), grid, dim3(256), 0, s, S, items, parts);
  else
    hipLaunchKernelGGL((k_rows<D, G, NV, false>), grid, dim3(256), 0, s, S, items, parts);
}

template <typename D, typename G>
hipError_t sums(const SumArgs &S, hipStream_t s) {
  const int v = (S.d + 7) / 8;
  const int parts = (v + 319) / 320;  // of a row, over at most five vectors of 8 columns per lane
  const int nv = (v + 64 * parts - 1) / (64 * parts);
  const long long items = S.accumulate ? S.n : S.vocab;
  if (items > 0) {
    switch (nv) {
      case 1: rows_nv<D, G, 1>(S, items, parts, s); break;
      case 2: rows_nv<D, G, 2>(S, items, parts, s); break;
      case 3: rows_nv<D, G, 3>(S, items, parts, s); break;
      case 4: rows_nv<D, G, 4>(S, items, parts, s); break;
      default: rows_nv<D, G, 5>(S, items, parts, s); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (S.n <= kChunk) return hipSuccess;  // no row can be long
  const unsigned chunks = (unsigned)((S.n + kChunk - 1) / kChunk);
  const dim3 g1(chunks, (unsigned)((v + 255) / 256)), g2(chunks, (unsigned)((v + 63) / 64));
  if (S.d % 8) {
    hipLaunchKernelGGL((k_long<D, true>), g1, dim3(256), 0, s, S);
    hipLaunchKernelGGL((k_join<G, true>), g2, dim3(kJoinWaves * 64), 0, s, S);
  } else {
    hipLaunchKernelGGL((k_long<D, false>), g1, dim3(256), 0, s, S);
    hipLaunchKernelGGL((k_join<G, false>), g2, dim3(kJoinWaves * 64), 0, s, S);
  }
  return hipGetLastError();
}

// The workspace of a gradient call, by offset.
struct GradWs {
  size_t key[2], pos[2], hist, seg, part, total;
};

GradWs grad_ws(long long n, int vocab, int d) {
  const SortPlan p = sort_plan(n, vocab);
  GradWs w;
  size_t off = 0;
  auto take = [&](size_t &at, size_t bytes) {
    at = off;
    off += (bytes + 255) & ~size_t(255);
  };
  for (int k = 0; k < 2; ++k) {
    take(w.key[k], (size_t)n * 4);
    take(w.pos[k], (size_t)n * 4);
  }
  take(w.hist, ((size_t)p.tiles << p.digit) * 4);
  take(w.seg, (size_t)vocab * sizeof(Run));
  take(w.part, n > kChunk ? (size_t)((n + kChunk - 1) / kChunk) * 2 * d * 4 : 0);
  w.total = off;
  return w;
}

}  // namespace

size_t embed_grad_ws_bytes(long long n, int vocab, int d) { return grad_ws(n, vocab, d).total; }

hipError_t launch_embed(const EmbedArgs &a, int E_f32, int x_f32, hipStream_t s) {
  if (a.ids.n <= 0) return hipSuccess;
  if (E_f32) return x_f32 ? embed<float, float>(a, s) : embed<float, bf16_t>(a, s);
  return x_f32 ? embed<bf16_t, float>(a, s) : embed<bf16_t, bf16_t>(a, s);
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, int dx_f32, int dE_f32, hipStream_t s) {
  const int n = a.ids.n;
  if (n <= 0 && a.accumulate) return hipSuccess;
  const SortPlan p = sort_plan(n, a.vocab);
  const GradWs w = grad_ws(n, a.vocab, a.d);
  char *ws = (char *)a.ws;
  SortArgs S{};
  S.ids = a.ids;
  S.vocab = a.vocab;
  S.bins = 1 << p.digit;
  S.tile = p.tile;
  S.tiles = p.tiles;
  S.hist = (uint32_t *)(ws + w.hist);
  S.seg = (Run *)(ws + w.seg);
  for (int k = 0; k < p.passes; ++k) {
    S.shift = k * p.digit;
    S.key_in = k ? (const uint32_t *)(ws + w.key[(k - 1) & 1]) : nullptr;
    S.pos_in = k ? (const uint32_t *)(ws + w.pos[(k - 1) & 1]) : nullptr;
    S.key_out = (uint32_t *)(ws + w.key[k & 1]);
    S.pos_out = (uint32_t *)(ws + w.pos[k & 1]);
    // the first pass also clears seg, with workgroups beyond the tiles' where the table is large
    int grid = p.tiles;
    const int clear = (a.vocab + kClearPerGroup - 1) / kClearPerGroup;
    if (k == 0 && clear > grid) grid = clear < kMaxTiles ? clear : kMaxTiles > grid ? kMaxTiles : grid;
    hipLaunchKernelGGL(k_sort_count, dim3(grid), dim3(kSortThreads), 0, s, S);
    if (!p.tiles) break;
    hipLaunchKernelGGL(k_sort_place, dim3(p.tiles), dim3(kSortThreads), 0, s, S);
  }
  SumArgs G{};
  G.dx = a.dx;
  G.dE = a.dE;
  G.key = S.key_out;
  G.pos = S.pos_out;
  G.seg = S.seg;
  G.part = (float *)(ws + w.part);
  G.n = n;
  G.vocab = a.vocab;
  G.d = a.d;
  G.accumulate = a.accumulate;
  G.scale = a.scale;
  if (n > 0)
    hipLaunchKernelGGL(k_segments, dim3((unsigned)((n + 255LL) / 256)), dim3(256), 0, s, G.key, n, a.vocab, S.seg);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (dx_f32) return dE_f32 ? sums<float, float>(G, s) : sums<float, bf16_t>(G, s);
  return dE_f32 ? sums<bf16_t, float>(G, s) : sums<bf16_t, bf16_t>(G, s);
}

// Token embedding with a scale, x[t] = scale * E[ids[t]], and its gradient,
// dE[v] = scale * sum of dx[t] over the tokens t with ids[t] = v. An id outside
// [0, vocab) gives a zero row and takes no gradient (the zero target rows of
// the layer follow the same reading).
//
// The gradient does not add with atomics, whose order would change its bits:
// the tokens are sorted by id, stably, so that each table row's tokens lie
// together in the order of their positions, and each row's columns are summed
// in fp32 in that order, by one thread each. Ids are skewed in real text, so a
// row of more than kChunk tokens is cut at multiples of kChunk sorted tokens;
// the pieces are summed side by side and joined in order, in fp64. The sort is
// a radix sort of (id, position) by counting: per pass, each workgroup counts
// its tile's digits, and then places its tokens from the counts of all tiles.
#include "embed.h"
#include "vec8.h"

namespace {

// x larger than this is written past the caches: the last level of them holds 256 MiB, and at half a GiB little of it
// would be left for the next kernel (measured at 168 MB and 1.3 GB, with nothing between)
constexpr double kStreamBytes = 512.0 * (1 << 20);
constexpr int kMaxTiles = 256;   // of a sort: a workgroup reads the counts of all of them
constexpr int kMinTile = 1024;   // tokens
constexpr int kMaxDigit = 9;     // bits
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kClearPerGroup = 2048;  // table rows whose segments one workgroup clears
static_assert(kMinTile == kSortThreads, "a token per thread");
constexpr int kSmallRounds = 4, kSmall = kSortThreads * kSmallRounds;  // tokens that one workgroup sorts by itself
constexpr int kSmallRows = 8191, kSmallWide = 3000;  // and of tables of more rows than kSmallRows
constexpr int kSmallClear = 16384;  // table rows whose segments one workgroup clears in passing
constexpr int kChunk = 32;       // sorted tokens of one piece of a long row

// ---- lookup ----

template <bool ONE, bool STREAM>
constexpr int kEmbedRows = ONE && STREAM ? 2 : 1;

// A workgroup takes one row or two neighbouring ones (ONE: their ids are the
// same for all threads and their addresses need no vector arithmetic), or, of
// narrow rows, `rpb` rows of `tr` threads. There is a workgroup for every row or
// two: a grid that keeps the card full and strides over the rows measured 470
// us on 131072 bf16 rows of 2560 into fp32 where this one takes 265 (1.52 GB:
// 5.7 TB/s), since rows that run at the same time then lie side by side in
// memory. STREAM: x is too large to be found in the caches later; its rows are
// written past them (342 us without; at 168 MB 60 us with it and 39 without),
// two at a time, so that their loads overlap (295 us one at a time, 332 four;
// within the caches one is as good or better). Writing x in pages of 4 KiB by
// threads that each find their row: 375 us and more.
template <typename E, typename X, bool R, bool ONE, bool STREAM>
__global__ __launch_bounds__(1024) void k_embed(EmbedArgs A, int tr, int rpb) {
  const int sub = ONE ? 0 : threadIdx.x / tr, d = A.d;
  // four columns of each half of an fp32 row: each store of a wave then covers whole cache lines (5% on rows that
  // stay in the caches)
  constexpr bool HALVES = !R && sizeof(X) == 4;
  constexpr int ROWS = kEmbedRows<ONE, STREAM>;
  const long long row0 = group_index() * rpb * ROWS + sub;
  const E *src[ROWS];
  bool on[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int id = row0 + k < A.ids.n ? A.ids.at((unsigned)(row0 + k)) : -1;
    on[k] = id >= 0 && id < A.vocab;
    src[k] = reinterpret_cast<const E *>(A.E) + (long long)(on[k] ? id : 0) * d;
  }
  for (int c8 = ONE ? threadIdx.x : threadIdx.x % tr; c8 * 8 < d; c8 += tr) {
    // the last columns of a ragged row: its last eight, some of which the neighbour writes too, to the same values
    const int c = R && c8 * 8 + 8 > d ? d - 8 : c8 * 8;
    Raw8<E> r[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
      r[k] = HALVES ? load_halves(src[k] + c8 * 4, d / 2, on[k]) : load_raw(src[k] + c, on[k]);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if (row0 + k >= A.ids.n) break;
      X *dst = reinterpret_cast<X *>(A.x) + (row0 + k) * d;
      float v[8];
      expand(r[k], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= A.scale;
      if constexpr (HALVES)
        store_halves<STREAM>(dst + c8 * 4, d / 2, v);
      else if constexpr (STREAM)
        stream_w(dst + c, true, v);
      else
        store_w(dst + c, true, v);
    }
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
  const uint32_t *key_in, *pos_in;  // NULL in the first pass: its counts read the ids, its positions are the tokens' own
  uint32_t *key_out, *pos_out;
  uint32_t *key_first;  // where the first pass's counts leave the keys: the ids are read once, so counts and places agree
  uint32_t *hist;  // [tiles][bins]
  Run *seg;        // [vocab], cleared by the first pass's counts
  __device__ __forceinline__ uint32_t key(int i) const {
    if (key_in) return key_in[i];
    const int id = ids.at((unsigned)i);
    return id >= 0 && id < vocab ? (uint32_t)id : (uint32_t)vocab;
  }
};

// seg of a table from `at` on, in steps
__device__ __forceinline__ void clear_runs(Run *seg, int vocab, long long at, long long step) {
  for (long long v = at; v < vocab; v += step) seg[v] = Run{0, 0};
}
__global__ __launch_bounds__(256) void k_clear_runs(Run *seg, int vocab) {
  clear_runs(seg, vocab, (long long)blockIdx.x * 256 + threadIdx.x, (long long)gridDim.x * 256);
}

// hist[tile][digit]: how often each digit occurs in the tile
__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs S) {
  __shared__ uint32_t cnt[1 << kMaxDigit];
  for (int i = threadIdx.x; i < S.bins; i += kSortThreads) cnt[i] = 0;
  if (!S.key_in)
    clear_runs(S.seg, S.vocab, (long long)blockIdx.x * kSortThreads + threadIdx.x, (long long)gridDim.x * kSortThreads);
  if ((int)blockIdx.x >= S.tiles) return;  // here to clear only
  __syncthreads();
  const long long t0 = (long long)blockIdx.x * S.tile;
  const int hi = (int)(t0 + S.tile < S.ids.n ? t0 + S.tile : S.ids.n);
  for (int i = (int)t0 + threadIdx.x; i < hi; i += kSortThreads) {
    const uint32_t key = S.key(i);
    if (!S.key_in) S.key_first[i] = key;
    atomicAdd(&cnt[(key >> S.shift) & (S.bins - 1)], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < S.bins; i += kSortThreads) S.hist[(long long)blockIdx.x * S.bins + i] = cnt[i];
}

// The place of a lane's token among the wave's: `next` holds where the wave's
// next token of each digit goes, and moves on. Tokens of one digit keep the
// order of their lanes.
__device__ __forceinline__ uint32_t place_of(uint32_t *next, int dg, int bins, bool in) {
  const int lane = threadIdx.x & 63;
  uint64_t same = __ballot(in);  // the lanes with the same digit
  for (int bit = 1; bit < bins; bit <<= 1) {
    const uint64_t one = __ballot(in && (dg & bit));
    same &= (dg & bit) ? one : ~one;
  }
  uint32_t at = 0;
  if (in) {
    const int first = __ffsll((unsigned long long)same) - 1;
    if (lane == first) at = atomicAdd(&next[dg], (uint32_t)__popcll(same));
    at = __shfl(at, first) + __popcll(same & ((1ull << lane) - 1));
  }
  return at;
}

// Turns next[wave][digit], how many tokens of each digit the waves have, into
// where their first ones go: behind the tokens of smaller digits and those of
// earlier waves. total: how many tokens of digit threadIdx.x there are in all,
// before: how many of them lie in front of this workgroup's.
__device__ __forceinline__ void first_places(uint32_t (*next)[1 << kMaxDigit], uint32_t *wsum, int bins, uint32_t total,
                                             uint32_t before) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, b = threadIdx.x;
  uint32_t inc = total;
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  if (b < bins) {
    uint32_t at = inc - total + before;
    for (int w = 0; w < wave; ++w) at += wsum[w];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = next[w][b];
      next[w][b] = at;
      at += c;
    }
  }
  __syncthreads();
}

// Places the tile's tokens: behind all tokens of a smaller digit, and those of
// the same digit in earlier tiles, earlier waves' parts of the tile (each wave
// owns a run of it) and earlier steps of the wave. ONCE: tiles of kMinTile, a
// token per thread, kept in registers. The counts of the tiles are the longest
// wait (they come from other dies): they are loaded many at a time, even and
// odd tiles by half the threads. 32768 tokens, 32 tiles: 7 us (with a quarter
// of the threads and four tokens each 11; with tiles of 4096 9).
template <bool ONCE>
__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortArgs S) {
  __shared__ uint32_t next[kSortWaves][1 << kMaxDigit];  // where a wave's next token of a digit goes
  __shared__ uint32_t odd[2][1 << kMaxDigit];            // totals and counts before this tile, of odd tiles
  __shared__ uint32_t wsum[kSortWaves];
  static_assert(kSortThreads == 2 << kMaxDigit, "a thread per digit and half of the tiles");
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const long long t0 = (long long)blockIdx.x * S.tile;
  const int run = S.tile / kSortWaves;
  const long long w0 = t0 + (long long)wave * run;
  const int lo = (int)(w0 < S.ids.n ? w0 : S.ids.n), hi = (int)(w0 + run < S.ids.n ? w0 + run : S.ids.n);
  uint32_t key = 0, pos = 0;
  auto load = [&](int i) {
    key = i < hi ? S.key(i) : 0;
    pos = i < hi && S.pos_in ? S.pos_in[i] : (uint32_t)i;
  };
  auto digit = [&]() { return (int)((key >> S.shift) & (S.bins - 1)); };
  if (ONCE) load(lo + lane);
  uint32_t total = 0, before = 0;
  const int b = threadIdx.x & ((1 << kMaxDigit) - 1), half = threadIdx.x >> kMaxDigit;
  if (b < S.bins) {
#pragma unroll 16
    for (int t = half; t < S.tiles; t += 2) {
      const uint32_t h = S.hist[(long long)t * S.bins + b];
      total += h;
      before += t < (int)blockIdx.x ? h : 0;
    }
  }
  for (int i = threadIdx.x; i < kSortWaves * S.bins; i += kSortThreads) next[i / S.bins][i % S.bins] = 0;
  if (half) {
    odd[0][b] = total;
    odd[1][b] = before;
    total = before = 0;
  }
  __syncthreads();
  if (!half) {
    total += odd[0][b];
    before += odd[1][b];
  }
  for (int i0 = lo; i0 < hi; i0 += 64) {
    if (!ONCE) load(i0 + lane);
    if (i0 + lane < hi) atomicAdd(&next[wave][digit()], 1u);
  }
  first_places(next, wsum, S.bins, total, before);
  for (int i0 = lo; i0 < hi; i0 += 64) {
    if (!ONCE) load(i0 + lane);
    const bool in = i0 + lane < hi;
    const uint32_t at = place_of(next[wave], digit(), S.bins, in);
    if (in) {
      S.key_out[at] = key;
      S.pos_out[at] = pos;
    }
  }
}

// What a chunk of kChunk sorted tokens holds of long rows (of more than kChunk
// tokens): the one it opens with, which may have begun earlier, and the one it
// closes with if that is another. A long row cannot lie inside a chunk, so
// there are no others.
struct Chunk {
  int v0, end0, starts0;  // table row (-1: none), end of its tokens in the chunk, and whether it begins with the chunk
  int v1, lo1;            // table row (-1: none) and the first of its tokens
};

// The runs that begin or end with sorted token i, and, in the first lane of
// each chunk, the chunk. A lane per token; `key` may lie in any memory.
static_assert(kChunk == 32, "half a wave's lanes are a chunk's tokens");
__device__ __forceinline__ void segment(const uint32_t *key, int n, int vocab, long long i, Run *seg, Chunk *chunks) {
  const bool in = i < n;
  const uint32_t k = in ? key[i] : 0;
  const bool head = in && (i == 0 || key[i - 1] != k);
  const bool tail = in && (i == n - 1 || key[i + 1] != k);
  if (head && k < (uint32_t)vocab) seg[k].start = (int)i;
  if (tail && k < (uint32_t)vocab) seg[k].end = (int)i + 1;
  const int half = threadIdx.x & 32;
  const uint32_t heads = (uint32_t)(__ballot(head) >> half), tails = (uint32_t)(__ballot(tail) >> half);
  if (!in || (threadIdx.x & 31)) return;
  const int a = (int)i, b = a + kChunk < n ? a + kChunk : n;
  Chunk c;
  c.starts0 = (int)(heads & 1);
  // the row the chunk opens with either goes on behind it, which takes more than kChunk tokens, or ends here, and is
  // long if the token kChunk before its last is its own
  c.end0 = tails ? a + __ffs((int)tails) : b;
  const bool long0 = !tails || (c.end0 > kChunk && key[c.end0 - 1 - kChunk] == k);
  c.v0 = k < (uint32_t)vocab && long0 ? (int)k : -1;
  c.v1 = -1;
  c.lo1 = 0;
  const uint32_t later = heads & ~1u;
  if (later) {
    const int lo = a + 31 - __clz((int)later);  // the row the chunk closes with
    const uint32_t k1 = key[lo];
    c.lo1 = lo;
    if (k1 < (uint32_t)vocab && lo + kChunk < n && key[lo + kChunk] == k1) c.v1 = (int)k1;
  }
  chunks[a / kChunk] = c;
}

__global__ __launch_bounds__(256) void k_segments(const uint32_t *key, int n, int vocab, Run *seg, Chunk *chunks) {
  segment(key, n, vocab, (long long)blockIdx.x * 256 + threadIdx.x, seg, chunks);
}

// The whole sort of up to kSmall tokens, and their segments, in one workgroup:
// one launch in place of five, which would be most of a short batch's time.
// CLEAR: it also clears seg, of a table that one workgroup clears sooner than a
// launch. Accumulating gradient calls in a captured graph, 256 columns, ids
// drawn with a share of 1 / rank, this way and by tiles: 512 rows, 2560 tokens
// 26.4 and 30.0 us, 4096 29.7 and 30.5; 4000 rows, 4096 tokens 30.2 both ways;
// 8000 rows, 3200 tokens 30.8 and 31.7, 4096 32.5 and 31.9. The keys of more
// rows than that have 14 bits or more, and placing them takes two more steps a
// pass: 16000 rows, 3000 tokens 31.0 and 31.8, 3500 32.9 and 32.0; 32000 rows,
// 2560 tokens 31.2 and 31.7, 3000 32.0 both ways, 4096 35.7 and 33.3; 151936
// rows, 3000 tokens 33.9 and 34.2, 3200 34.3 and 33.6. Eight tokens per thread
// are too many for any table: 6216 tokens, 1024 columns, 29.8 and 25.8 us with
// 512 rows, 50.5 and 42.0 with 32000.
template <bool CLEAR>
__global__ __launch_bounds__(kSortThreads) void k_sort_small(SortArgs S, int passes, int digit, Chunk *chunks) {
  __shared__ uint32_t skey[kSmall], spos[kSmall];
  __shared__ uint32_t next[kSortWaves][1 << kMaxDigit];
  __shared__ uint32_t wsum[kSortWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = S.ids.n;
  if (CLEAR) clear_runs(S.seg, S.vocab, threadIdx.x, kSortThreads);
  // of a wave: up to kSmallRounds steps
  const int run = (n + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64, lo = wave * run;
  uint32_t key[kSmallRounds], pos[kSmallRounds];
#pragma unroll
  for (int r = 0; r < kSmallRounds; ++r) {
    const int i = lo + r * 64 + lane;
    key[r] = r * 64 < run && i < n ? S.key(i) : 0;
    pos[r] = (uint32_t)i;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * digit;
    for (int i = threadIdx.x; i < kSortWaves * S.bins; i += kSortThreads) next[i / S.bins][i % S.bins] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r)
      if (r * 64 < run && lo + r * 64 + lane < n) atomicAdd(&next[wave][(key[r] >> shift) & (S.bins - 1)], 1u);
    __syncthreads();
    uint32_t total = 0;
    if ((int)threadIdx.x < S.bins)
      for (int w = 0; w < kSortWaves; ++w) total += next[w][threadIdx.x];
    first_places(next, wsum, S.bins, total, 0);
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) {
      if (r * 64 >= run) break;
      const bool in = lo + r * 64 + lane < n;
      const uint32_t to = place_of(next[wave], (int)((key[r] >> shift) & (S.bins - 1)), S.bins, in);
      if (in) {
        skey[to] = key[r];
        spos[to] = pos[r];
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) {
      const int i = lo + r * 64 + lane;
      if (r * 64 < run && i < n) {
        key[r] = skey[i];
        pos[r] = spos[i];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kSmallRounds; ++r) {
    if (r * 64 >= run) break;
    const int i = lo + r * 64 + lane;
    if (i < n) {
      S.key_out[i] = key[r];
      S.pos_out[i] = pos[r];
    }
    segment(skey, n, S.vocab, i, S.seg, chunks);
  }
}

// ---- sums ----

struct SumArgs {
  const void *dx;
  void *dE;
  const uint32_t *key, *pos;  // sorted
  const Run *seg;
  const Chunk *chunks;
  float *part;  // [chunks][2][d]
  int n, vocab, d, accumulate;
  int nchunks;  // 0 where no row can be long
  float scale;
};

// The scaled sum of eight columns into the table's gradient. `first`: a
// thread at the end of a ragged row owns its columns from there on only.
template <bool STREAM, typename G>
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
  if constexpr (STREAM)
    stream_w(p, true, s);
  else
    store_w(p, true, s);
}

// Adds eight columns of the sorted tokens lo .. hi-1, in order; the loads of
// eight tokens run at once.
template <typename D, bool HALVES>
__device__ __forceinline__ void add_rows(const SumArgs &S, int c, int lo, int hi, float (&acc)[8]) {
  const D *dx = reinterpret_cast<const D *>(S.dx) + c;
  for (int t = lo; t < hi; t += 8) {
    Raw8<D> r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool on = t + k < hi;
      const D *q = dx + (long long)S.pos[on ? t + k : lo] * S.d;
      r[k] = HALVES ? load_halves(q, S.d / 2, on) : load_raw(q, on);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float v[8];
      expand(r[k], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[j];
    }
  }
}

// Neighbouring workgroups run on different dies, and cache lines and pages that
// two of them write cost; here each die takes 64 neighbours at a time (of n).
__device__ __forceinline__ long long beside(long long w, long long n) {
  constexpr int kDies = 8, kRun = 64;
  const long long base = w / (kDies * kRun) * (kDies * kRun);
  if (base + kDies * kRun > n) return w;
  const int k = (int)(w - base);
  return base + k % kDies * kRun + k / kDies;
}

// Items: first the chunks, whose long rows' sums go to part[chunk][0 or 1];
// then the table rows, or, when the sums are added to dE, the sorted tokens,
// which count if they are the first of their row. A table row's tokens are
// summed in order; long rows are left to their chunks and k_join. A workgroup
// takes an item (ONE: what it reads to find its tokens is the same for all
// threads), or, of narrow rows, rpb items of tr threads.
//
// Most rows of a large table do not occur and only take zeros, so the launch is
// bound by writing: 151936 fp32 rows of 2560 (1.56 GB) from 32768 bf16 tokens
// take 307 us (5.6 TB/s). A fill in the same rows takes 285, one in pages of
// 4 KiB 227, but sums by pages, where each thread has to find its row, 395.
// What matters is HALVES: a thread has four columns of each half of an fp32
// row, so that each store of a wave covers whole cache lines (with eight in a
// row, written past the caches: 620 us); STREAM, as in the lookup (355 us
// without); and the order (325 us without). Several rows per workgroup, side
// by side or apart, gain nothing.
template <typename D, typename G, bool R, bool ONE, bool STREAM, bool HALVES>
__global__ __launch_bounds__(1024) void k_sums(SumArgs S, long long items, int tr, int rpb) {
  const int sub = ONE ? 0 : threadIdx.x / tr, d = S.d;
  const int t0 = ONE ? threadIdx.x : threadIdx.x % tr;
  long long w = group_index();
  if (STREAM) w = beside(w, (long long)gridDim.x * gridDim.y);
  const long long g = w * rpb + sub;
  if (g < S.nchunks) {
    const Chunk k = S.chunks[g];
    for (int c8 = t0; c8 * 8 < d; c8 += tr) {
      const int at = R && c8 * 8 + 8 > d ? d - 8 : c8 * 8;
      if (k.v0 >= 0) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        add_rows<D, false>(S, at, (int)g * kChunk, k.end0, acc);
        store_w(S.part + g * 2 * d + at, true, acc);
      }
      if (k.v1 >= 0) {
        const int b = ((int)g + 1) * kChunk;
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        add_rows<D, false>(S, at, k.lo1, b < S.n ? b : S.n, acc);
        store_w(S.part + (g * 2 + 1) * d + at, true, acc);
      }
    }
    return;
  }
  long long v = g - S.nchunks;
  if (v >= items) return;
  if (S.accumulate) {
    const long long i = v;
    v = S.key[i];
    if (v >= S.vocab || (i > 0 && S.key[i - 1] == (uint32_t)v)) return;
  }
  const Run run = S.seg[v];
  if (run.end - run.start > kChunk) return;
  G *out = reinterpret_cast<G *>(S.dE) + v * d;
  for (int c8 = t0; c8 * 8 < d; c8 += tr) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if constexpr (HALVES) {
      add_rows<D, true>(S, c8 * 4, run.start, run.end, acc);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] *= S.scale;
      store_halves<STREAM>(out + c8 * 4, d / 2, acc);
    } else {
      const int at = R && c8 * 8 + 8 > d ? d - 8 : c8 * 8;
      add_rows<D, false>(S, at, run.start, run.end, acc);
      put<STREAM>(out + at, R ? c8 * 8 - at : 0, S.accumulate, S.scale, acc);
    }
  }
}

// A long row from its pieces: workgroup (chunk, 512 columns) for the long row
// that begins in the chunk, each wave a run of the pieces, the waves' sums
// joined in order. Eight pieces are added in fp32 and their sums in fp64, since
// a batch may hold one id (a padding, say) in most of its up to 2^27 tokens: so
// many pieces one behind the other in fp32 lose up to half of a piece's last
// place each, together 2e-4 of the row at 2^22 tokens and some percent at 2^27.
// Each eight pieces are under way at once: a padding id in 131072 bf16 tokens of
// 2560 takes 389 us with its sort and sums (pieces as the compiler orders their
// loads 557, all in fp64 420 and more, all in fp32 450).
constexpr int kJoinWaves = 8, kJoinStep = 8;  // waves, and pieces of a step
template <typename G, bool R>
__global__ __launch_bounds__(kJoinWaves * 64) void k_join(SumArgs S) {
  __shared__ double sum[kJoinWaves][64][9];
  const Chunk chunk = S.chunks[blockIdx.x];
  const int d = S.d, i = chunk.v1 >= 0 ? 1 : 0;
  const int v = i ? chunk.v1 : chunk.starts0 ? chunk.v0 : -1;
  if (v < 0) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = (blockIdx.y * 64 + lane) * 8;
  const int at = R && c + 8 > d ? d - 8 : c;
  const int last = (S.seg[v].end - 1) / kChunk;  // pieces: (blockIdx.x, i), then (j, 0) up to the last chunk
  const int pieces = last - (int)blockIdx.x + 1, run = (pieces + kJoinWaves - 1) / kJoinWaves;
  double acc[8] = {0., 0., 0., 0., 0., 0., 0., 0.};
  if (c < d) {
    const int p0 = wave * run, p1 = p0 + run < pieces ? p0 + run : pieces;
    auto piece = [&](int p) {
      return load_raw(S.part + (((long long)blockIdx.x + p) * 2 + (p == 0 ? i : 0)) * d + at, true);
    };
    int p = p0;
    for (; p + kJoinStep <= p1; p += kJoinStep) {
      Raw8<float> r[kJoinStep];
#pragma unroll
      for (int k = 0; k < kJoinStep; ++k) r[k] = piece(p + k);
      __builtin_amdgcn_sched_barrier(0);  // all of them under way before the first is waited for
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x = r[0].f[j];
#pragma unroll
        for (int k = 1; k < kJoinStep; ++k) x += r[k].f[j];
        acc[j] += (double)x;
      }
    }
    for (; p < p1; ++p) {
      const Raw8<float> r = piece(p);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += (double)r.f[j];
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
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = (float)acc[j];
  put<false>(reinterpret_cast<G *>(S.dE) + (long long)v * d + at, R ? c - at : 0, S.accumulate, S.scale, s);
}

// ---- which instance ----

// threads of a row of d, and rows of a workgroup
struct RowThreads {
  int tr, rpb;
};
RowThreads row_threads(int d) {
  const int v = (d + 7) / 8;
  int tr = 8;
  while (tr < v && tr < 64) tr *= 2;
  if (v > 64) tr = v >= 1024 ? 1024 : (v + 63) / 64 * 64;
  return {tr, tr <= 64 ? 256 / tr : 1};
}

template <typename E, typename X, bool R, bool ONE, bool STREAM>
void embed_launch(const EmbedArgs &a, int tr, int rpb, hipStream_t s) {
  const int rows = rpb * kEmbedRows<ONE, STREAM>;
  const dim3 grid = group_grid((a.ids.n + rows - 1LL) / rows);
  hipLaunchKernelGGL((k_embed<E, X, R, ONE, STREAM>), grid, dim3(tr * rpb), 0, s, a, tr, rpb);
}

template <typename E, typename X, bool R, bool ONE>
void embed_form(const EmbedArgs &a, int tr, int rpb, hipStream_t s) {
  // not ragged rows: parts of cache lines written past the caches cost more (491 MB: 187 us, 129 through them)
  if (!R && (double)a.ids.n * a.d * sizeof(X) > kStreamBytes)
    embed_launch<E, X, R, ONE, !R>(a, tr, rpb, s);
  else
    embed_launch<E, X, R, ONE, false>(a, tr, rpb, s);
}

template <typename E, typename X>
hipError_t embed(const EmbedArgs &a, hipStream_t s) {
  const auto [tr, rpb] = row_threads(a.d);
  if (rpb > 1)
    a.d % 8 ? embed_form<E, X, true, false>(a, tr, rpb, s) : embed_form<E, X, false, false>(a, tr, rpb, s);
  else
    a.d % 8 ? embed_form<E, X, true, true>(a, tr, rpb, s) : embed_form<E, X, false, true>(a, tr, rpb, s);
  return hipGetLastError();
}

template <typename D, typename G, bool R, bool ONE>
void sums_form(const SumArgs &S, int tr, int rpb, hipStream_t s) {
  const long long items = S.accumulate ? (long long)S.n : S.vocab;
  const dim3 grid = group_grid((S.nchunks + items + rpb - 1) / rpb), block(tr * rpb);
  constexpr bool halves = !R && sizeof(G) == 4;
  if (!R && !S.accumulate && (double)S.vocab * S.d * sizeof(G) > kStreamBytes)
    hipLaunchKernelGGL((k_sums<D, G, R, ONE, !R, halves>), grid, block, 0, s, S, items, tr, rpb);
  else if (halves && !S.accumulate)
    hipLaunchKernelGGL((k_sums<D, G, R, ONE, false, halves>), grid, block, 0, s, S, items, tr, rpb);
  else
    hipLaunchKernelGGL((k_sums<D, G, R, ONE, false, false>), grid, block, 0, s, S, items, tr, rpb);
}

template <typename D, typename G>
hipError_t sums(const SumArgs &S, hipStream_t s) {
  const RowThreads m = row_threads(S.d);
  if (m.rpb > 1)
    S.d % 8 ? sums_form<D, G, true, false>(S, m.tr, m.rpb, s) : sums_form<D, G, false, false>(S, m.tr, m.rpb, s);
  else
    S.d % 8 ? sums_form<D, G, true, true>(S, m.tr, m.rpb, s) : sums_form<D, G, false, true>(S, m.tr, m.rpb, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !S.nchunks) return e;
  const dim3 grid((unsigned)S.nchunks, (unsigned)((S.d + 511) / 512));
  if (S.d % 8)
    hipLaunchKernelGGL((k_join<G, true>), grid, dim3(kJoinWaves * 64), 0, s, S);
  else
    hipLaunchKernelGGL((k_join<G, false>), grid, dim3(kJoinWaves * 64), 0, s, S);
  return hipGetLastError();
}

// The workspace of a gradient call, by offset.
struct GradWs {
  size_t key[2], pos[2], hist, seg, chunks, part, total;
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
  const size_t chunks = (size_t)((n + kChunk - 1) / kChunk);
  take(w.chunks, chunks * sizeof(Chunk));
  take(w.part, n > kChunk ? chunks * 2 * d * 4 : 0);
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
  const bool small = n > 0 && n <= (a.vocab <= kSmallRows ? kSmall : kSmallWide);
  if (small) {
    S.key_out = (uint32_t *)(ws + w.key[0]);
    S.pos_out = (uint32_t *)(ws + w.pos[0]);
    Chunk *chunks = (Chunk *)(ws + w.chunks);
    if (a.vocab <= kSmallClear) {
      hipLaunchKernelGGL(k_sort_small<true>, dim3(1), dim3(kSortThreads), 0, s, S, p.passes, p.digit, chunks);
    } else {
      const int clear = (a.vocab + kClearPerGroup - 1) / kClearPerGroup;
      hipLaunchKernelGGL(k_clear_runs, dim3(clear < kMaxTiles ? clear : kMaxTiles), dim3(256), 0, s, S.seg, a.vocab);
      hipLaunchKernelGGL(k_sort_small<false>, dim3(1), dim3(kSortThreads), 0, s, S, p.passes, p.digit, chunks);
    }
  }
  for (int k = 0; k < p.passes && !small; ++k) {
    S.shift = k * p.digit;
    S.key_in = k ? (const uint32_t *)(ws + w.key[(k - 1) & 1]) : nullptr;
    S.pos_in = k ? (const uint32_t *)(ws + w.pos[(k - 1) & 1]) : nullptr;
    S.key_out = (uint32_t *)(ws + w.key[k & 1]);
    S.pos_out = (uint32_t *)(ws + w.pos[k & 1]);
    S.key_first = (uint32_t *)(ws + w.key[1]);
    // the first pass also clears seg, with workgroups beyond the tiles' where the table is large
    int grid = p.tiles;
    const int clear = (a.vocab + kClearPerGroup - 1) / kClearPerGroup;
    if (k == 0 && clear > grid) grid = clear < kMaxTiles ? clear : kMaxTiles > grid ? kMaxTiles : grid;
    hipLaunchKernelGGL(k_sort_count, dim3(grid), dim3(kSortThreads), 0, s, S);
    if (!p.tiles) break;
    if (k == 0) S.key_in = S.key_first;
    if (p.tile == kMinTile)
      hipLaunchKernelGGL(k_sort_place<true>, dim3(p.tiles), dim3(kSortThreads), 0, s, S);
    else
      hipLaunchKernelGGL(k_sort_place<false>, dim3(p.tiles), dim3(kSortThreads), 0, s, S);
  }
  SumArgs G{};
  G.dx = a.dx;
  G.dE = a.dE;
  G.key = S.key_out;
  G.pos = S.pos_out;
  G.seg = S.seg;
  G.chunks = (const Chunk *)(ws + w.chunks);
  G.nchunks = n > kChunk ? (n + kChunk - 1) / kChunk : 0;
  G.part = (float *)(ws + w.part);
  G.n = n;
  G.vocab = a.vocab;
  G.d = a.d;
  G.accumulate = a.accumulate;
  G.scale = a.scale;
  if (n > 0 && !small)
    hipLaunchKernelGGL(k_segments, dim3((unsigned)((n + 255LL) / 256)), dim3(256), 0, s, G.key, n, a.vocab, S.seg,
                       (Chunk *)(ws + w.chunks));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (dx_f32) return dE_f32 ? sums<float, float>(G, s) : sums<float, bf16_t>(G, s);
  return dE_f32 ? sums<bf16_t, float>(G, s) : sums<bf16_t, bf16_t>(G, s);
}

// The products of operands whose rows start on 16 bytes: tiles that go from
// memory straight into LDS.
//
// A workgroup of WI x WJ waves computes a tile of D; each wave 16 FI x 16 FJ of
// it with v_mfma_f32_16x16x32_bf16, or in fp32 with four v_mfma_f32_16x16x4_f32
// for every one of those. Tiles of 256 x 256 take eight waves of 128 x 64, one
// workgroup per CU; tiles of 128 x 128 four of 64 x 64, two workgroups per CU;
// tiles of 64 x 64 four of 32 x 32, three or four per CU. k runs in slabs of one
// 128-byte line (64 k in bf16, 32 in fp32): a load instruction moves eight
// lines into LDS (16 bytes per lane), SLABS of them are held, and the loads of
// slab n + SLABS are issued behind the MFMAs of slab n's second half, into the
// buffer that half has just finished reading. The fragments of the next half
// and of the second half of rows are read behind MFMAs already queued.
//
// An operand that lies by rows is held as [rows][k], the eight 16-byte chunks
// of a row permuted by swz(row), which leaves the fragments' reads free of bank
// conflicts. One that lies transposed is held as it lies, in blocks of [k][a
// line of rows]: in bf16 permuted by zsw(k), its fragments from transposing
// reads (ds_read_b64_tr_b16); in fp32 unpermuted, its fragments read element by
// element, four lanes to a bank, which costs less than the four times longer
// MFMAs leave. Rows, k and transposed rows past an operand's end are addressed
// behind the end of its buffer descriptor, which reads zero; columns past a
// transposed operand's row read the next row, and only reach elements of D that
// are not stored.
//
// The epilogue takes a wave's sums through LDS, 32 j at a time, so that a lane
// holds eight consecutive i and a row's stores cover whole lines.
//
// Measured: 32768 x 9728 x 2560 in bf16 1.30 ms, 1250 TFLOP/s, the MFMA pipes
// busy 63 % of the cycles at the 1.75 GHz that the power limit leaves; a slab's
// LDS traffic takes as long as its MFMAs. fp32, 8192 x 1024 x 4096: 508 us, 135
// TFLOP/s (566 for the general kernel), 1233 x 1024 x 512: 23.7 (25.1). Tiles of
// 64 against the larger ones, bf16: 32 x 9728 x 2560 17 us (23), 256 x 2560 x
// 2560 15 (21), a weight's gradient of 512 x 512 over 4096 rows 16 (19); but
// 4096 x 1024 x 2048 33 (22).
#include <type_traits>

#include "lds_dma.h"
#include "linear_dev.h"
#include "tiles.h"

namespace {

template <typename T>
constexpr int SK = 128 / (int)sizeof(T);  // k per slab: one line
template <typename T>
constexpr int EL = 16 / (int)sizeof(T);  // elements of a 16-byte chunk

template <typename T>
__device__ __forceinline__ int lds_off(int r, int c) { return r * SK<T> + (c ^ swz(r)) * EL<T>; }
// 16 bytes per lane from memory to LDS. TRACKED: as the compiler's own. With
// transposing reads it would then wait for every load in flight before each of
// them (1.29 -> 1.64 ms for 32768 x 9728 x 2560), so there the load is one that
// it does not track, ordered by the kernel's counted waits and barriers alone.
template <bool TRACKED>
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rs, void *lds, uint32_t voff) {
  if constexpr (TRACKED)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)lds, 16, voff, 0, 0, 0);
  else
    dma16_untracked(rs, lds, voff);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, bytes > 0 ? bytes : 0, kBufferFlags);
}

// The loads of one operand's tile by one wave: 8 N of its rows (or, transposed, 8 N of a block's k), 1 KB each. The
// chunks' permutations depend on the load only through its parity.
template <typename T, bool TRANS, int N>
struct Loads {
  static constexpr int ES = (int)sizeof(T);
  const T *seg[2];  // first row of this wave's matrix, per segment; transposed: first column of its block
  int ld;
  int span;  // bytes from there to the end of the wave's rows; transposed: of the columns before its block
  long long nk;
  uint32_t vo[N];
  int k[2];  // of the lane's piece in a slab (by rows), for even and odd loads
  int lds0;  // element offset of the wave's share

  // by rows: row0 is the operand's row that the wave's first tile row holds; transposed: the tile's first column
  __device__ __forceinline__ void init(const void *s0, const void *s1, long long ld_, long long row0, long long nrows,
                                       long long nk_, int w, int lane) {
    ld = (int)ld_;
    nk = nk_;
    lds0 = w * 8 * N * SK<T>;
    if constexpr (TRANS) {
      // blocks are SK rows of k by SK columns
      const int k0 = w * 8 * N % SK<T>;
      const long long col = row0 + w * 8 * N / SK<T> * SK<T>;
      seg[0] = (const T *)s0 + col;
      seg[1] = (const T *)s1 + col;
      span = (int)col * ES;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int kr = k0 + 8 * n + (lane >> 3);
        vo[n] = (uint32_t)(kr * ld * ES + (((lane & 7) ^ (ES == 2 ? zsw(kr) : 0)) << 4));
      }
    } else {
      seg[0] = (const T *)s0 + row0 * ld;
      seg[1] = (const T *)s1 + row0 * ld;
      const long long rows = nrows - row0;
      span = (int)(rows < 0 ? 0 : rows > 8 * N ? 8 * N : rows) * ld * ES;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int r = 8 * n + (lane >> 3), c = (lane & 7) ^ swz(r);
        if (n < 2) k[n] = c * EL<T>;
        vo[n] = (uint32_t)(r * ld * ES + c * 16);
      }
    }
  }
  struct Pre {
    __amdgpu_buffer_rsrc_t rs;
    bool past[2];  // the lane's piece lies past the last k
  };
  __device__ __forceinline__ Pre prep(int sg, long long k0) const {
    Pre p;
    const T *s = sg ? seg[1] : seg[0];
    const long long left = nk - k0;
    if constexpr (TRANS) {
      // from the slab's first row to the end of its last: rows past the last k lie behind it
      p.rs = rsrc(s + k0 * ld, (int)(left < SK<T> ? left : SK<T>) * ld * ES - span);
    } else {
      // behind the last k of a row lies the next one
      p.rs = rsrc(s + k0, span - (int)k0 * ES);
      p.past[0] = k[0] >= left;
      p.past[1] = k[1] >= left;
    }
    return p;
  }
  template <bool TRACKED>
  __device__ __forceinline__ void issue(const Pre &p, T *tile, int n) const {
    uint32_t v = vo[n];
    if (!TRANS && p.past[n & 1]) v = kOutOfRange;
    dma16<TRACKED>(p.rs, tile + lds0 + n * 8 * SK<T>, v);
  }
};

template <int FI_, int FJ_, int WI_, int WJ_, int SLABS_, int PER_CU_>
struct Shape {
  static constexpr int FI = FI_, FJ = FJ_, WI = WI_, WJ = WJ_, NW = WI * WJ, SLABS = SLABS_, PER_CU = PER_CU_;
  static constexpr int TI = 16 * FI * WI, TJ = 16 * FJ * WJ;
  static constexpr int N = TI / (8 * NW);  // loads of a wave per operand and slab
  static_assert(TI == TJ && N % 2 == 0, "square tiles; a wave's rows are whole periods of the chunks' permutation");
  static constexpr int THREADS = 64 * NW;
  static constexpr int SLAB = (TI + TJ) * 128;  // bytes
  static constexpr int PITCH = 16 * FI + 4;     // of the epilogue's rows, fp32
  static constexpr int RING = SLABS * SLAB, OUT = NW * 32 * PITCH * 4;
  static constexpr int SMEM = RING > OUT ? RING : OUT;
};
using Big = Shape<8, 4, 2, 4, 2, 1>;
template <typename T>
using Small = Shape<4, 4, 2, 2, 2, 2>;
// Tiles of 64: bf16 waits for memory and gains by a third slab (256 x 2560 x 2560 15 us, 22 with two); fp32 waits for its
// MFMAs and gains by more workgroups (4096 x 1024 x 1024 70 us, 75 with three slabs).
template <typename T>
using Tiny = Shape<2, 2, 2, 2, sizeof(T) == 2 ? 3 : 2, sizeof(T) == 2 ? 3 : 4>;

// Every wave's loads but the last LATER have landed, and its reads of LDS are done.
template <int LATER>
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_s_waitcnt(wait_imm(LATER));
  asm volatile("s_barrier" ::: "memory");
}
// 16 bytes per lane of 16 rows: eight bf16 k, or four fp32 ones of the sixteen that half a slab has.
template <typename T>
struct Fragment;
template <>
struct Fragment<bf16_t> {
  typedef bf16x8 type;
};
template <>
struct Fragment<float> {
  typedef f32x4 type;
};
// N fragments (16 rows each) of the tile rows from r0, half h of the slab.
template <typename T, bool TRANS, int N>
__device__ __forceinline__ void read(typename Fragment<T>::type (&f)[N], const T *tile, int r0, int h, int lane) {
  if constexpr (!TRANS) {
    const int c = 4 * h + (lane >> 4);
#pragma unroll
    for (int x = 0; x < N; ++x)
      f[x] = *reinterpret_cast<const typename Fragment<T>::type *>(tile + lds_off<T>(r0 + 16 * x + (lane & 15), c));
  } else if constexpr (sizeof(T) == 2) {
    const int lo = z_lane_off(lane);
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int r = r0 + 16 * x;  // the lane's offset is even in 16-byte chunks, so fragment r / 16 of a block is a XOR
      const bf16_t *p = tile + (r >> 6) * 4096 + h * 2048 + (lo ^ (((r >> 4) & 3) << 4));
      const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)p);
      const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)(p + 256));
      f[x] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  } else {
    const int k = 16 * h + 4 * (lane >> 4);
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int r = r0 + 16 * x + (lane & 15);
#pragma unroll
      for (int s = 0; s < 4; ++s) f[x][s] = tile[(r >> 5) * 1024 + (k + s) * 32 + (r & 31)];
    }
  }
}
// One fragment of rows times N of columns. The fp32 products that add to one sum are N apart.
template <int N>
__device__ __forceinline__ void multiply(f32x4 (&acc)[N], const bf16x8 &a, const bf16x8 (&b)[N]) {
#pragma unroll
  for (int y = 0; y < N; ++y) acc[y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[y], acc[y], 0, 0, 0);
}
template <int N>
__device__ __forceinline__ void multiply(f32x4 (&acc)[N], const f32x4 &a, const f32x4 (&b)[N]) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int y = 0; y < N; ++y) acc[y] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[y][s], acc[y], 0, 0, 0);
}

// Bands of four: the 32 tiles of an XCD at a time are 4 x 8. (32768 x 9728 x 2560: 1263 us; 1295 in bands of 8, 1355 of
// 16, and 2 and 3 cost products of wide outputs 1 to 2 %.)
constexpr int kBand = 4;

template <class S, typename T, typename O, bool AT, bool BT, bool PAIR>
__global__ __launch_bounds__(S::THREADS, S::PER_CU * S::NW / 4) void k_dense(GemmArgs g, int nti, int ntj, Parts parts) {
  __shared__ __attribute__((aligned(16))) char smem[S::SMEM];
  constexpr int FI = S::FI, FJ = S::FJ, HF = FI / 2, HALF = 8 * FI;  // HALF: a pair's rows of one matrix in a wave
  constexpr int WIDE = PAIR ? S::TI / 2 : S::TI;
  const int per_split = nti * ntj * g.batch;
  const int logical = xcd_tile(blockIdx.x, gridDim.x);
  const int split = logical / per_split, rest = logical % per_split, z = rest / (nti * ntj);
  int tx, ty;
  band_tile(rest % (nti * ntj), nti, ntj, kBand, tx, ty);
  const long long i0 = (long long)tx * WIDE, j0 = (long long)ty * S::TJ;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wi = w % S::WI, wj = w / S::WI;

  constexpr int N = S::N, RW = 8 * N;  // rows of the tile that a wave loads
  Loads<T, AT, N> la;
  Loads<T, BT, N> lb;
  if constexpr (PAIR) {
    // rows RW w .. of the tile: their group of 2 HALF, the matrix and the row within it
    const int q = w * RW % (2 * HALF);
    const long long row = i0 + w * RW / (2 * HALF) * HALF + q % HALF;
    la.init(g.a[q / HALF], g.a[q / HALF], g.lda, row, g.ni, g.nk, w, lane);
  } else {
    la.init(g.a[0], g.a[1], g.lda, AT ? i0 : i0 + w * RW, g.ni, g.nk, w, lane);
  }
  lb.init(g.b[z], g.b[1], g.ldb, BT ? j0 : j0 + w * RW, g.nj, g.nk, w, lane);

  const int per = (int)((g.nk + SK<T> - 1) / SK<T>), slabs = per * g.segments;
  const int first = (int)((long long)slabs * split / parts.splits);
  const int end = (int)((long long)slabs * (split + 1) / parts.splits);

  f32x4 acc[FI][FJ];
#pragma unroll
  for (int a = 0; a < FI; ++a)
#pragma unroll
    for (int b = 0; b < FJ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  constexpr int SLABS = S::SLABS;
  // of two buffers the slab's parity names one, which costs 1 % less than counting turns
  auto buffer = [](int sl, int turn) { return SLABS == 2 ? sl & 1 : turn; };
  auto tile_a = [&](int buf) { return reinterpret_cast<T *>(smem + buf * S::SLAB); };
  auto tile_b = [&](int buf) { return reinterpret_cast<T *>(smem + buf * S::SLAB + S::TI * 128); };
  struct Pre {
    typename Loads<T, AT, N>::Pre a;
    typename Loads<T, BT, N>::Pre b;
  };
  auto prep = [&](int sl) {
    const int sg = sl >= per;
    const long long k0 = (long long)(sl - sg * per) * SK<T>;
    return Pre{la.prep(sg, k0), lb.prep(sg, k0)};
  };
  auto issue = [&](const Pre &p, int buf, int n) {  // load n of 2 N
    if (n < N)
      la.template issue<!AT && !BT>(p.a, tile_a(buf), n);
    else
      lb.template issue<!AT && !BT>(p.b, tile_b(buf), n - N);
  };
  typename Fragment<T>::type lo[HF], hi[HF], fb[2][FJ];
  const int ra = wi * 16 * FI, rb = wj * 16 * FJ;

  // Half H of slab sl, which buffer cb holds and nb the next. On entry lo and fb[H] hold its fragments of the first half
  // of rows and of the columns; on exit those of the next half. REFILL: slab sl + SLABS is there to be loaded.
  auto stage = [&](int sl, int cb, int nb, auto half, auto refill) {
    constexpr int H = decltype(half)::value;
    constexpr bool REFILL = decltype(refill)::value;
    read<T, AT, HF>(hi, tile_a(cb), ra + 16 * HF, H, lane);
    pin();
    multiply(acc[0], lo[0], fb[H]);
    pin();
    Pre p;
    if (H == 1) {
      // slab sl + 1 has landed (while others are refilled, those behind it may be on their way), and no wave reads slab
      // sl any more
      meet<REFILL ? (SLABS - 2) * 2 * N : 0>();
      if (REFILL) p = prep(sl + SLABS);
    }
    pin();
#pragma unroll
    for (int x = 1; x < FI; ++x) {
      multiply(acc[x], x < HF ? lo[x % HF] : hi[x % HF], fb[H]);
      if (x == HF) {
        pin();
        // past the last slab this reads what the next buffer holds, and nothing uses it
        read<T, AT, HF>(lo, tile_a(H ? nb : cb), ra, H ^ 1, lane);
        read<T, BT, FJ>(fb[H ^ 1], tile_b(H ? nb : cb), rb, H ^ 1, lane);
      }
      if (REFILL) {
#pragma unroll
        for (int n = (x - 1) * 2 * N / (FI - 1); n < x * 2 * N / (FI - 1); ++n) issue(p, cb, n);
      }
      pin();
    }
  };
  using T0 = std::integral_constant<int, 0>;
  using T1 = std::integral_constant<int, 1>;
  if (first < end) {
#pragma unroll
    for (int u = 0; u < SLABS; ++u) {
      if (first + u >= end) continue;
      const Pre p = prep(first + u);
#pragma unroll
      for (int n = 0; n < 2 * N; ++n) issue(p, buffer(first + u, u), n);
    }
    if (first + SLABS <= end)
      meet<(SLABS - 1) * 2 * N>();
    else
      meet<0>();
    read<T, AT, HF>(lo, tile_a(buffer(first, 0)), ra, 0, lane);
    read<T, BT, FJ>(fb[0], tile_b(buffer(first, 0)), rb, 0, lane);
    int sl = first, turn = 0;
    auto slab = [&](auto refill) {
      const int next = turn + 1 == SLABS ? 0 : turn + 1;
      const int cb = buffer(sl, turn), nb = buffer(sl + 1, next);
      stage(sl, cb, nb, T0{}, std::false_type{});
      stage(sl, cb, nb, T1{}, refill);
      turn = next;
    };
    for (; sl + SLABS < end; ++sl) slab(std::true_type{});
    for (; sl < end; ++sl) slab(std::false_type{});
  }
  __syncthreads();  // the ring is free

  // Epilogue: the wave's sums of 32 j as [j][i], then eight i of one j per lane. A lane keeps its i throughout.
  float *stg = reinterpret_cast<float *>(smem) + w * 32 * S::PITCH;
  constexpr int LANES = (PAIR ? HALF : 2 * HALF) / 8;  // lanes to a row
  constexpr int STEP = 64 / LANES;                     // rows at a time
  const int ii = lane % LANES * 8;
  const long long i = i0 + wi * (PAIR ? HALF : 2 * HALF) + ii;
  const int left = clamp8(g.ni - i);
  constexpr int ROUNDS = 32 / STEP;
  const O *res = PAIR ? nullptr : reinterpret_cast<const O *>(g.res[z]);
#pragma unroll
  for (int q = 0; q < FJ / 2; ++q) {
    const long long jq = j0 + rb + 32 * q;
    Raw8<O> old[PAIR ? 1 : ROUNDS];  // the residual, on its way while the sums go through LDS
    if constexpr (!PAIR) {
      if (res && parts.splits == 1) {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
          const long long j = jq + r * STEP + lane / LANES;
          old[r] = load_some(res + j * g.ldo + i, j < g.nj ? left : 0);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y)
        *reinterpret_cast<f32x4 *>(stg + (16 * y + (lane & 15)) * S::PITCH + 16 * x + 4 * (lane >> 4)) = acc[x][2 * q + y];
    // the wave's own LDS writes and reads run in order
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int row = r * STEP + lane / LANES;
      const long long j = jq + row;
      float v[8], u[8];
      __builtin_memcpy(v, __builtin_assume_aligned(stg + row * S::PITCH + ii, 16), 32);
      if constexpr (PAIR) __builtin_memcpy(u, __builtin_assume_aligned(stg + row * S::PITCH + HALF + ii, 16), 32);
      if (parts.splits > 1) {
        float *p = parts.at + (((long long)split * per_split + (long long)z * nti * ntj + (long long)ty * nti + tx) * S::TJ +
                               rb + 32 * q + row) * S::TI + wi * 2 * HALF + ii;
        __builtin_memcpy(__builtin_assume_aligned(p, 16), v, 32);
        if constexpr (PAIR) __builtin_memcpy(__builtin_assume_aligned(p + HALF, 16), u, 32);
      } else if (j < g.nj && left > 0) {
        if constexpr (PAIR)
          finish_pair<T, true>(g, i, j, left, v, u);
        else
          finish<T, O, true>(g, z, i, j, left, v, &old[r]);
      }
      end_of_stores();
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

template <class S, typename T, typename O, bool AT, bool BT, bool PAIR>
hipError_t run(const GemmArgs &g, const GemmForm &f, int splits, hipStream_t s) {
  const int wide = PAIR ? S::TI / 2 : S::TI;
  const long long ti = (g.ni + wide - 1) / wide, tj = (g.nj + S::TJ - 1) / S::TJ;
  if (ti * tj == 0) return hipSuccess;
  if (ti * tj * g.batch * splits * S::THREADS >= 1LL << 32) return hipErrorInvalidConfiguration;
  const Parts parts{(float *)g.ws, splits, S::TI, S::TJ, 8 * S::FI};
  hipLaunchKernelGGL((k_dense<S, T, O, AT, BT, PAIR>), dim3((unsigned)(ti * tj * g.batch * splits)), dim3(S::THREADS), 0,
                     s, g, (int)ti, (int)tj, parts);
  return splits > 1 ? launch_join(g, f, ti, tj, parts, s) : hipGetLastError();
}

template <class S, typename T, typename O>
hipError_t run(const GemmArgs &g, const GemmForm &f, int splits, hipStream_t s) {
  if (f.pair) return run<S, T, T, false, false, true>(g, f, splits, s);
  if (!f.a_trans) return run<S, T, O, false, false, false>(g, f, splits, s);
  return f.b_trans ? run<S, T, T, true, true, false>(g, f, splits, s) : run<S, T, T, true, false, false>(g, f, splits, s);
}
template <template <typename> class S>
hipError_t run(const GemmArgs &g, const GemmForm &f, int splits, hipStream_t s) {
  if (f.f32) return run<S<float>, float, float>(g, f, splits, s);
  return f.out_f32 ? run<S<bf16_t>, bf16_t, float>(g, f, splits, s) : run<S<bf16_t>, bf16_t, bf16_t>(g, f, splits, s);
}

}  // namespace

long long dense_tiles(const GemmArgs &g, const GemmForm &f, int tile) {
  const int wide = f.pair ? tile / 2 : tile;
  return (g.ni + wide - 1) / wide * ((g.nj + tile - 1) / tile) * g.batch;
}

// Rows are whole 16-byte pieces, k fits an int, and the tiles a launch, whose threads count in 32 bits: 2^23 tiles of 64
// and as many larger ones as hold them. Split tiles are fewer by far: their sums may take 512 MB (choose()).
bool dense_sizes(const GemmArgs &g, const GemmForm &f) {
  const int el = f.f32 ? 4 : 8;
  return g.lda % el == 0 && g.ldb % el == 0 && dense_tiles(g, f, 64) <= (1LL << 23) && g.nk > 0 &&
         g.nk * g.segments <= (1LL << 34);
}
hipError_t launch_dense(const GemmArgs &g, const GemmForm &f, int tile, int splits, hipStream_t s) {
  if (tile == 256 && !f.f32)
    return f.out_f32 ? run<Big, bf16_t, float>(g, f, splits, s) : run<Big, bf16_t, bf16_t>(g, f, splits, s);
  return tile == 128 ? run<Small>(g, f, splits, s) : run<Tiny>(g, f, splits, s);
}

// What the kernels whose tiles go from memory straight into LDS share
// (kernels_bf16.hip, kernels_dense.hip): buffer descriptors, the layouts of a
// tile in LDS, waits, and the order of tiles.
#pragma once

#include "common.h"

constexpr uint32_t kBufferFlags = 0x00020000u;  // raw buffer descriptor word 3 on the gfx9 family
constexpr uint32_t kOutOfRange = 0x80000000u;   // offset past num_records: the load returns zero

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// The eight 16-byte chunks of each 128-byte LDS row are XOR-swizzled; with
// this pattern the fragment reads (32 consecutive rows, one chunk) are free of
// bank conflicts, also while LDS-DMA writes land (measured with rocprofv3).
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// Chunk swizzle of a tile held transposed ([k][64 rows]): k row r holds logical
// chunk c at c ^ zsw(r). A transposing read of one 16-lane group g covers 4 consecutive
// k rows r0 + 8g .. +3 and one pair of adjacent chunks in each; the LDS
// serves 32 lanes (two groups, 8 rows apart) at a time. zsw(r) =
// 2*((r%4) ^ (r/8 % 2)) gives the 4 rows of one parity (rows of a 128-byte
// stride alternate between the two halves of the 64 banks) of the two groups
// the four disjoint chunk pairs of that half, so the read is free of bank
// conflicts.
__device__ __forceinline__ int zsw(int r) { return ((r & 3) ^ ((r >> 3) & 1)) << 1; }

// A fragment of such a tile: rows 16gi + l%16 of a 64-row block (lane l), k
// 8(l/16) .. +7 of half a slab, from two transposing reads (ds_read_b64_tr_b16)
// of 4 k rows each. In each 16-lane group g, lane t addresses k row
// 8g + t/4 (+4 for the second read), columns 4(t%4) .. +3 of the fragment's
// 16 (one 8-byte piece), and receives column t of the 4 rows. This is lane
// l's element offset for gi = 0; the chunk pair of fragment gi is gi
// further on, which in the swizzled row is `^ (gi << 4)` (zsw is even, so
// the XOR leaves the 8-byte half within the chunk alone).
__device__ __forceinline__ int z_lane_off(int lane) {
  const int t = lane & 15, g = lane >> 4;
  const int krow = 8 * g + (t >> 2);
  const int chunk = ((t & 3) >> 1) ^ zsw(krow);
  return krow * 64 + chunk * 8 + 4 * (t & 1);
}

// s_waitcnt immediate (gfx9): vmcnt(n), expcnt unchanged, lgkmcnt(0).
constexpr unsigned wait_imm(int n) { return (unsigned)((n & 15) | 0x70 | (((n >> 4) & 3) << 14)); }

// Keep the compiler from moving instructions across this point.
__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0); }

// Workgroups of a launch are handed to the 8 XCDs round-robin (workgroup n to
// XCD n % 8), and each XCD has its own L2. Renumber them so that XCD k works
// through one contiguous range of the logical tile order: the workgroups
// resident on an XCD at one time are then neighbours in that order and share
// operand tiles in its L2. A bijection on [0, N).
constexpr int kXcds = 8;
__device__ __forceinline__ int xcd_tile(int n, int N) {
  const int xcd = n % kXcds, m = n / kXcds;
  const int q = N / kXcds, r = N % kXcds;
  return xcd * q + (xcd < r ? xcd : r) + m;
}

// Logical tile t of an nx x ny grid, in bands of H rows along y; inside a band
// y runs fastest, so H consecutive tiles share one x and nx*H consecutive tiles
// cover the band. The last band may be shorter.
__device__ __forceinline__ void band_tile(int t, int nx, int ny, int H, int &x, int &y) {
  const int full = ny / H, per = H * nx;
  const int band = t / per;
  const int h = band < full ? H : ny - full * H;
  const int r = t - band * per;
  x = r / h;
  y = band * H + r % h;
}

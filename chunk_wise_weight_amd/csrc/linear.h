// The matrix products of the plain layers (kernels_linear.hip): launch arguments.
#pragma once

#include "common.h"

// One product D[i][j] = sum_k A(i, k) B(j, k) and what becomes of it, element (i, j) at out[j * ldo + i]. An operand
// is held by rows (element (i, k) at a[i * lda + k]) or transposed (at a[k * lda + i]).
//
//   segments : k runs through the two pairs a[0], b[0] and a[1], b[1] one after the other, nk each
//   batch    : two products, a[0] with b[0] into out[0] and a[0] with b[1] into out[1]
//   pair     : A's rows are those of two matrices a[0], a[1], products g and u: out[0] = act(g) u, and pre[0], pre[1]
//              receive g and u
//
// Without pair: p = D + bias[0], pre[0] receives p, out = res + scale * act(p), res of out's type.
struct GemmArgs {
  const void *a[2], *b[2];
  long long lda, ldb;
  long long ni, nj, nk;
  int segments, batch;
  const void *bias[2];  // of the operands' type
  const void *res[2];
  void *out[2];
  void *pre[2];  // of the operands' type, laid out like out
  long long ldo;
  float scale;
  int act;  // TTT_ACT_*
  void *ws;  // gemm_ws_bytes
};

struct GemmForm {
  bool f32;               // the operands' type
  bool a_trans, b_trans;  // held transposed
  bool pair;
  bool out_f32;
};

// Workspace of a product by its sizes (ni, nj, nk, segments, batch) and form alone, wherever its arrays lie.
size_t gemm_ws_bytes(const GemmArgs &g, const GemmForm &f);
// How it runs where its arrays start on 16 bytes: on a kernel of TTT_KERNEL_*, tiles of `tile` (0: none), k in `splits`
// parts, with `copies` operands copied first.
struct GemmPlan {
  int kernel, tile, splits, copies;
};
GemmPlan gemm_plan(const GemmArgs &g, const GemmForm &f);
hipError_t launch_gemm(const GemmArgs &g, const GemmForm &f, hipStream_t s);

// Sums of a part of k, fp32, for k_join: [splits][batch][tiles][tj][ti], tiles in the order j, i, of ti rows of A (with
// a pair `half` of the first matrix, then the matching `half` of the second, and so on) and tj of B.
struct Parts {
  float *at;
  int splits;  // 1: none, the product is finished at once
  int ti, tj, half;
};

// The second launch of a split product (kernels_linear.hip); tiles: ti by tj of them per batch.
hipError_t launch_join(const GemmArgs &g, const GemmForm &f, long long ti, long long tj, const Parts &p, hipStream_t s);

// Forward products of few rows (kernels_few.hip).
bool few_sizes(const GemmArgs &g, const GemmForm &f);
hipError_t launch_few(const GemmArgs &g, const GemmForm &f, hipStream_t s);

// Operands whose rows start on 16 bytes (kernels_dense.hip): sizes that allow it, the launch with tiles of `tile` x
// `tile` (64, 128 or, in bf16, 256), and its workgroups (tiles times batch). k past nk in the last 16 bytes of a row of
// an operand held by rows is zero.
bool dense_sizes(const GemmArgs &g, const GemmForm &f);
long long dense_tiles(const GemmArgs &g, const GemmForm &f, int tile);
hipError_t launch_dense(const GemmArgs &g, const GemmForm &f, int tile, int splits, hipStream_t s);

// q = scale * dy * act'(p) (p NULL: scale * dy), rounded to out's type, and its column sums. dy, p, u: [rows][n]; out,
// out2: rows of n at ldo, which is n or n rounded up to eight, and then zeros behind.
// gated (u not NULL): out2 = dy * act(p), out = dy * u * act'(p).
struct ActGradArgs {
  const void *dy, *p, *u;
  void *out, *out2;  // nullable: only the sums are wanted
  float *sum, *sum2;  // [n] fp32, nullable
  float *part;        // act_grad_ws_bytes(rows, n, gated), with sum
  long long rows, n, ldo;
  float scale;
  int act, accumulate;  // accumulate: the sums are added to sum, sum2
  bool dy_f32, f32;     // types of dy; of p, u, out, out2
};
size_t act_grad_ws_bytes(long long rows, long long n, bool gated);
hipError_t launch_act_grad(const ActGradArgs &a, hipStream_t s);

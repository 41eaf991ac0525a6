// Arguments of the norm kernels (kernels_norm.hip), as the entry points fill them.
#pragma once

#include "common.h"

struct NormArgs {
  long long rows;
  int d;
  float eps, alpha, beta;
  const void *h;       // residual stream [rows][d]: h of the forward; o (the stream after the block) of a gradient
  const void *y;       // the block's output [rows][d]; NULL: no block (a norm before the first one)
  const void *w;       // gain of the norm after the block [d], or NULL (ones)
  const void *gate;    // [d] or [rows][d], or NULL
  const void *w_next;  // gain of the norm before a block [d], or NULL (ones)
  int p_f32;           // w, w_next and a gate per channel are fp32 (else bf16)
  int token_gate;      // the gate is [rows][d], of y's type
  // forward
  void *o;  // [rows][d], of h's type
  void *x;  // [rows][d]; NULL: no norm before a block
  // gradient
  const void *dx;           // gradient of x, or NULL
  const void *dh_in;        // gradient of o from the rows after, or NULL
  void *dh, *dy, *dgate_t;  // gradients of h, y and a gate per token
  float *dw, *dgate_c, *dw_next;  // gradients of the parameters, or NULL
  float *part;              // workspace
  float shrink, grow, mean;  // of a row's sums: 2^-k, 2^k, and what a sum of shrunk squares is divided by for their
                             // mean, 4^-k d; set by the launchers
};

// Types of one call: residual stream, block output, block input (1: fp32, 0: bf16).
struct NormTypes {
  int h, y, x;
};

hipError_t launch_norm_fwd(const NormArgs &a, NormTypes t, hipStream_t s);
// post: a block came before (y, dy); next: the stream went on through a norm (dx)
hipError_t launch_norm_bwd(const NormArgs &a, NormTypes t, bool post, bool next, hipStream_t s);
// bytes of workspace of a gradient call
size_t norm_ws_bytes(long long rows, int d);

// Arguments of the embedding kernels (kernels_embed.hip), as the entry points fill them.
#pragma once

#include "common.h"

// The ids of a call: B rows of T, ld apart; token t is ids[t / T * ld + t % T].
struct TokenIds {
  const int32_t *ids;
  long long ld;
  int T;   // at least 1 where n > 0
  int n;   // B * T, 0 .. 2^27
  __device__ __forceinline__ int at(unsigned t) const {
    const unsigned b = t / (unsigned)T;
    return ids[b * ld + (t - b * (unsigned)T)];
  }
};

// x[t] = scale * E[ids[t]]
struct EmbedArgs {
  TokenIds ids;
  const void *E;
  void *x;
  int vocab, d;
  float scale;
};

// dE[v] (+)= scale * sum of dx[t] over ids[t] = v
struct EmbedGradArgs {
  TokenIds ids;
  const void *dx;
  void *dE;
  int vocab, d, accumulate;
  float scale;
  void *ws;
};

hipError_t launch_embed(const EmbedArgs &a, int E_f32, int x_f32, hipStream_t s);
hipError_t launch_embed_grad(const EmbedGradArgs &a, int dx_f32, int dE_f32, hipStream_t s);
size_t embed_grad_ws_bytes(long long n, int vocab, int d);

// C ABI of the operators around the layer: argument checks and launches. No
// call allocates, keeps state or waits.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <vector>

#include "../../include/ttt.h"
#include "embed.h"
#include "errors.h"
#include "grads.h"
#include "norm.h"

namespace {

constexpr int kMaxWidth = 65536;
constexpr long long kMaxRows = 0x7fffffffLL;
constexpr long long kMaxTokens = 1LL << 27;
constexpr int kMaxVocab = 1 << 30;

bool known(ttt_dtype t) { return t == TTT_F32 || t == TTT_BF16; }
size_t size_of(ttt_dtype t) { return t == TTT_BF16 ? 2 : 4; }

// An array of a call: its bytes, and the size of one element.
struct Span {
  const char *name;
  const void *p;
  size_t bytes, elem;
};

bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const char *x = (const char *)a.p, *y = (const char *)b.p;
  return x < y + b.bytes && y < x + a.bytes;
}

// Outputs against inputs and one another. in_place: pairs (output, input) that
// may be the same array.
struct Pair {
  const void *out, *in;
};
int check_spans(const char *where, std::initializer_list<Span> in, std::initializer_list<Span> out,
                std::initializer_list<Pair> in_place) {
  for (const Span &s : in)
    if ((uintptr_t)s.p % s.elem) return ttt_fail(TTT_E_ARG, "%s: %s is not aligned to its elements", where, s.name);
  for (const Span *o = out.begin(); o != out.end(); ++o) {
    if ((uintptr_t)o->p % o->elem) return ttt_fail(TTT_E_ARG, "%s: %s is not aligned to its elements", where, o->name);
    for (const Span &s : in) {
      if (!overlap(*o, s)) continue;
      bool ok = false;
      for (const Pair &p : in_place) ok = ok || (p.out == o->p && p.in == s.p && o->p == s.p && o->bytes == s.bytes);
      if (!ok) return ttt_fail(TTT_E_ARG, "%s: %s overlaps %s", where, o->name, s.name);
    }
    for (const Span *q = out.begin(); q != o; ++q)
      if (overlap(*o, *q)) return ttt_fail(TTT_E_ARG, "%s: %s overlaps %s", where, o->name, q->name);
  }
  return TTT_OK;
}

int check_norm(const char *where, ttt_dtype h, ttt_dtype y, ttt_dtype x, ttt_dtype w, bool post, bool next, float alpha,
               float beta, float eps, int64_t rows, int d) {
  if (!known(h) || !known(w) || (post && !known(y)) || (next && !known(x)))
    return ttt_fail(TTT_E_DTYPE, "%s: unknown dtype", where);
  if (post && y == TTT_F32 && h == TTT_BF16)
    return ttt_fail(TTT_E_DTYPE, "%s: an fp32 y needs an fp32 residual stream", where);
  if (next && x == TTT_F32 && (h == TTT_BF16 || (post && y == TTT_BF16)))
    return ttt_fail(TTT_E_DTYPE, "%s: an fp32 x needs fp32 inputs", where);
  if (d < 8 || d > kMaxWidth) return ttt_fail(TTT_E_SHAPE, "%s: d must be in [8, %d], got %d", where, kMaxWidth, d);
  if (rows < 0 || rows > kMaxRows)
    return ttt_fail(TTT_E_SHAPE, "%s: rows must be in [0, 2^31), got %lld", where, (long long)rows);
  if (!(eps >= 1e-30f) || !std::isfinite(eps))
    return ttt_fail(TTT_E_ARG, "%s: eps must be finite, at least 1e-30", where);
  if (!std::isfinite(alpha) || !std::isfinite(beta))
    return ttt_fail(TTT_E_ARG, "%s: alpha, beta must be finite", where);
  return TTT_OK;
}

int check_gate(const char *where, const void *gate, int kind, int64_t rows) {
  if (kind != TTT_GATE_NONE && kind != TTT_GATE_CHANNEL && kind != TTT_GATE_TOKEN)
    return ttt_fail(TTT_E_ARG, "%s: unknown gate kind %d", where, kind);
  if (kind != TTT_GATE_NONE && !gate && (kind == TTT_GATE_CHANNEL || rows > 0))
    return ttt_fail(TTT_E_NULL, "%s: gate is NULL", where);
  return TTT_OK;
}

size_t gate_bytes(int kind, int64_t rows, int d, size_t token, size_t channel) {
  return kind == TTT_GATE_TOKEN ? (size_t)rows * d * token : kind == TTT_GATE_CHANNEL ? (size_t)d * channel : 0;
}

NormTypes types(ttt_dtype h, ttt_dtype y, ttt_dtype x) { return NormTypes{h == TTT_F32, y == TTT_F32, x == TTT_F32}; }

int check_ws(const char *where, const void *ws, size_t have, size_t need) {
  if (!ws) return ttt_fail(TTT_E_NULL, "%s: the workspace is NULL", where);
  if ((uintptr_t)ws % 16) return ttt_fail(TTT_E_ARG, "%s: the workspace must be 16-byte aligned", where);
  if (have < need) return ttt_fail(TTT_E_SHAPE, "%s: needs %zu bytes of workspace, got %zu", where, need, have);
  return TTT_OK;
}

int check_tokens(const char *where, int B, int T, int64_t ids_ld, int vocab, int d, float scale) {
  if (d < 8 || d > kMaxWidth) return ttt_fail(TTT_E_SHAPE, "%s: d must be in [8, %d], got %d", where, kMaxWidth, d);
  if (vocab < 1 || vocab > kMaxVocab)
    return ttt_fail(TTT_E_SHAPE, "%s: vocab must be in [1, 2^30], got %d", where, vocab);
  if (B < 0 || T < 0 || (long long)B * T > kMaxTokens)
    return ttt_fail(TTT_E_SHAPE, "%s: B and T must not be negative and B * T at most 2^27", where);
  if (ids_ld < T || ids_ld > (1LL << 40)) return ttt_fail(TTT_E_SHAPE, "%s: ids_ld must be at least T", where);
  if (!std::isfinite(scale)) return ttt_fail(TTT_E_ARG, "%s: scale must be finite", where);
  return TTT_OK;
}

size_t ids_bytes(int B, int T, int64_t ids_ld) {
  return (long long)B * T ? ((size_t)(B - 1) * ids_ld + T) * sizeof(int32_t) : 0;
}

// ---- many tensors ----

constexpr int kMaxTensors = 1 << 20;
constexpr long long kMaxNumel = 1LL << 40;  // of all tensors: their chunks count in 32 bits
// gradients of more bytes than this are read and written past the caches, of which the last level holds 256 MiB
// (measured at 140 MB and 2.1 GB, with nothing between)
constexpr long long kStreamGrads = 512LL << 20;

// the workgroups' sums and, before them, the factor
size_t grad_ws(int n) { return ((size_t)kGradGroups + n / kGradTable + 2) * sizeof(double); }

int check_grads(const char *where, const void *const *grads, const int64_t *numel, const int32_t *dt, int n,
                const float *norm, const void *ws, size_t ws_bytes) {
  if (n < 0 || n > kMaxTensors) return ttt_fail(TTT_E_SHAPE, "%s: n must be in [0, 2^20], got %d", where, n);
  if (n > 0 && (!grads || !numel || !dt)) return ttt_fail(TTT_E_NULL, "%s: grads, numel or dt is NULL", where);
  if (!norm) return ttt_fail(TTT_E_NULL, "%s: norm is NULL", where);
  if ((uintptr_t)norm % 4) return ttt_fail(TTT_E_ARG, "%s: norm is not aligned to its elements", where);
  const int rc = check_ws(where, ws, ws_bytes, grad_ws(n));
  if (rc) return rc;
  long long total = 0;
  for (int i = 0; i < n; ++i) {
    if (!known((ttt_dtype)dt[i])) return ttt_fail(TTT_E_DTYPE, "%s: tensor %d has an unknown dtype", where, i);
    if (numel[i] < 0 || numel[i] > kMaxNumel || (total += numel[i]) > kMaxNumel)
      return ttt_fail(TTT_E_SHAPE, "%s: tensor %d has %lld elements; together at most 2^40 are taken", where, i,
                      (long long)numel[i]);
    if (numel[i] > 0 && !grads[i]) return ttt_fail(TTT_E_NULL, "%s: tensor %d is NULL", where, i);
    if ((uintptr_t)grads[i] % size_of((ttt_dtype)dt[i]))
      return ttt_fail(TTT_E_ARG, "%s: tensor %d is not aligned to its elements", where, i);
  }
  return TTT_OK;
}

// Where outputs and workspace lie: each overlaps nothing but, in place, its own gradient.
struct Extent {
  uintptr_t lo, hi;
  bool out;
};
int check_extents(const char *where, std::vector<Extent> &e) {
  std::sort(e.begin(), e.end(), [](const Extent &a, const Extent &b) { return a.lo < b.lo; });
  uintptr_t any = 0, outs = 0;  // ends of what came before
  for (const Extent &x : e) {
    if (x.lo < outs || (x.out && x.lo < any)) return ttt_fail(TTT_E_ARG, "%s: an output overlaps another array", where);
    any = std::max(any, x.hi);
    if (x.out) outs = std::max(outs, x.hi);
  }
  return TTT_OK;
}

// The tables of a launch, empty tensors left out and tensors that follow one
// another in memory (views of one buffer), with their outputs, taken as one:
// 2000 gradients of 1000 values in one buffer take 5 us so and 97 one by one.
// The norm's are made without outputs (NULL), so that its sum, which follows
// the cuts, does not change its last bit with where the outputs lie.
std::vector<GradTable> grad_tables(const void *const *grads, const int64_t *numel, const int32_t *dt, int n,
                                   void *const *out) {
  struct One {
    const char *g;
    char *o;
    long long n;
    int f32;
  };
  std::vector<One> all;
  all.reserve(n);
  for (int i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    const int f32 = dt[i] == TTT_F32;
    const One x{(const char *)grads[i], out ? (char *)out[i] : (char *)grads[i], (long long)numel[i], f32};
    if (!all.empty()) {
      One &p = all.back();
      const long long bytes = p.n * (p.f32 ? 4 : 2);
      if (p.f32 == x.f32 && p.g + bytes == x.g && p.o + bytes == x.o) {
        p.n += x.n;
        continue;
      }
    }
    all.push_back(x);
  }
  std::vector<GradTable> tables;
  for (size_t i = 0; i < all.size(); ++i) {
    if (tables.empty() || tables.back().n == kGradTable) {
      tables.emplace_back();
      tables.back().n = 0;
      tables.back().first[0] = 0;
    }
    GradTable &t = tables.back();
    const long long chunk = kGradBytes / (all[i].f32 ? 4 : 2), chunks = (all[i].n + chunk - 1) / chunk;
    t.g[t.n] = all[i].g;
    t.out[t.n] = all[i].o;
    t.tail[t.n] = (uint32_t)(all[i].n - (chunks - 1) * chunk);
    t.f32[t.n] = (uint8_t)all[i].f32;
    t.first[t.n + 1] = t.first[t.n] + (uint32_t)chunks;
    ++t.n;
  }
  return tables;
}

// Norm of the tables and, with `clip`, the scaling of its tables by it.
int run_grads(const char *where, const std::vector<GradTable> &tables, const std::vector<GradTable> *clip, float tau,
              float *norm, void *ws, hipStream_t s) {
  GradFactor *factor = (GradFactor *)ws;
  double *part = (double *)ws + 1;
  long long chunks = 0;
  for (const GradTable &t : tables) chunks += t.first[t.n];
  const bool stream = chunks * kGradBytes > kStreamGrads;
  int n = 0;
  for (const GradTable &t : tables) {
    // its share of kGradGroups
    const long long c = t.first[t.n], most = std::max(1LL, kGradGroups * c / chunks);
    const int groups = (int)std::min(c, most);
    const int rc = ttt_launched(launch_grad_squares(t, part + n, groups, stream, s), where);
    if (rc) return rc;
    n += groups;
  }
  int rc = ttt_launched(launch_grad_norm(part, n, tau, norm, clip ? factor : nullptr, s), where);
  if (!clip) return rc;
  for (const GradTable &t : *clip) {
    if (rc) break;
    rc = ttt_launched(launch_grad_scale(t, factor, stream, s), where);
  }
  return rc;
}

}  // namespace

extern "C" {

int ttt_norm_pre(const void *h, ttt_dtype h_dt, const void *w, ttt_dtype w_dt, float eps, int64_t rows, int d, void *x,
                 ttt_dtype x_dt, void *hip_stream) {
  static const char *kWhere = "ttt_norm_pre";
  int rc = check_norm(kWhere, h_dt, h_dt, x_dt, w_dt, false, true, 1.f, 1.f, eps, rows, d);
  if (rc) return rc;
  if (rows > 0 && (!h || !x)) return ttt_fail(TTT_E_NULL, "%s: h or x is NULL", kWhere);
  const size_t n = (size_t)rows * d;
  rc = check_spans(kWhere, {{"h", h, n * size_of(h_dt), size_of(h_dt)}, {"w", w, d * size_of(w_dt), size_of(w_dt)}},
                   {{"x", x, n * size_of(x_dt), size_of(x_dt)}}, {});
  if (rc) return rc;
  rc = ttt_check_device();
  if (rc || rows == 0) return rc;
  NormArgs a{};
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  a.alpha = a.beta = 1.f;
  a.h = h;
  a.w_next = w;
  a.p_f32 = w_dt == TTT_F32;
  a.x = x;
  return ttt_launched(launch_norm_fwd(a, types(h_dt, h_dt, x_dt), (hipStream_t)hip_stream), kWhere);
}

int ttt_norm_post(const void *h, ttt_dtype h_dt, const void *y, ttt_dtype y_dt, const void *w, const void *gate,
                  int gate_kind, const void *w_next, ttt_dtype w_dt, float alpha, float beta, float eps, int64_t rows,
                  int d, void *o, void *x, ttt_dtype x_dt, void *hip_stream) {
  static const char *kWhere = "ttt_norm_post";
  int rc = check_norm(kWhere, h_dt, y_dt, x_dt, w_dt, true, x != nullptr, alpha, beta, eps, rows, d);
  if (!rc) rc = check_gate(kWhere, gate, gate_kind, rows);
  if (rc) return rc;
  if (rows > 0 && (!h || !y || !o)) return ttt_fail(TTT_E_NULL, "%s: h, y or o is NULL", kWhere);
  const size_t n = (size_t)rows * d, ws = size_of(w_dt);
  const size_t ge = gate_kind == TTT_GATE_TOKEN ? size_of(y_dt) : ws;
  if (gate_kind == TTT_GATE_NONE) gate = nullptr;
  rc = check_spans(kWhere,
                   {{"h", h, n * size_of(h_dt), size_of(h_dt)},
                    {"y", y, n * size_of(y_dt), size_of(y_dt)},
                    {"w", w, d * ws, ws},
                    {"gate", gate, gate_bytes(gate_kind, rows, d, size_of(y_dt), ws), ge},
                    {"w_next", w_next, d * ws, ws}},
                   {{"o", o, n * size_of(h_dt), size_of(h_dt)}, {"x", x, n * size_of(x_dt), x ? size_of(x_dt) : 1}},
                   {{o, h}});
  if (rc) return rc;
  rc = ttt_check_device();
  if (rc || rows == 0) return rc;
  NormArgs a{};
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  a.alpha = alpha;
  a.beta = beta;
  a.h = h;
  a.y = y;
  a.w = w;
  a.gate = gate;
  a.token_gate = gate_kind == TTT_GATE_TOKEN;
  a.w_next = w_next;
  a.p_f32 = w_dt == TTT_F32;
  a.o = o;
  a.x = x;
  return ttt_launched(launch_norm_fwd(a, types(h_dt, y_dt, x_dt), (hipStream_t)hip_stream), kWhere);
}

int ttt_norm_ws_bytes(int64_t rows, int d, size_t *bytes) {
  if (!bytes) return ttt_fail(TTT_E_NULL, "ttt_norm_ws_bytes: bytes is NULL");
  const int rc =
      check_norm("ttt_norm_ws_bytes", TTT_F32, TTT_F32, TTT_F32, TTT_F32, true, true, 1.f, 1.f, 1.f, rows, d);
  if (rc) return rc;
  *bytes = norm_ws_bytes(rows, d);
  return TTT_OK;
}

int ttt_norm_pre_grad(const void *dx, ttt_dtype x_dt, const void *h, ttt_dtype h_dt, const void *w, ttt_dtype w_dt,
                      const void *dh_in, float eps, int64_t rows, int d, void *dh, float *dw, void *ws, size_t ws_bytes,
                      void *hip_stream) {
  static const char *kWhere = "ttt_norm_pre_grad";
  int rc = check_norm(kWhere, h_dt, h_dt, x_dt, w_dt, false, true, 1.f, 1.f, eps, rows, d);
  if (rc) return rc;
  if (rows > 0 && (!dx || !h || !dh)) return ttt_fail(TTT_E_NULL, "%s: dx, h or dh is NULL", kWhere);
  if (dw && (rc = check_ws(kWhere, ws, ws_bytes, norm_ws_bytes(rows, d)))) return rc;
  const size_t n = (size_t)rows * d, hs = size_of(h_dt);
  rc = check_spans(kWhere,
                   {{"dx", dx, n * size_of(x_dt), size_of(x_dt)},
                    {"h", h, n * hs, hs},
                    {"w", w, d * size_of(w_dt), size_of(w_dt)},
                    {"dh_in", dh_in, n * hs, hs}},
                   {{"dh", dh, n * hs, hs},
                    {"dw", dw, (size_t)d * 4, 4},
                    {"ws", dw ? ws : nullptr, norm_ws_bytes(rows, d), 4}},
                   {{dh, dh_in}});
  if (rc) return rc;
  rc = ttt_check_device();
  if (rc) return rc;
  NormArgs a{};
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  a.alpha = a.beta = 1.f;
  a.h = h;
  a.w_next = w;
  a.p_f32 = w_dt == TTT_F32;
  a.dx = dx;
  a.dh_in = dh_in;
  a.dh = dh;
  a.dw_next = dw;
  a.part = dw ? (float *)ws : nullptr;
  return ttt_launched(launch_norm_bwd(a, types(h_dt, h_dt, x_dt), false, true, (hipStream_t)hip_stream), kWhere);
}

int ttt_norm_post_grad(const void *dh_in, const void *dx, ttt_dtype x_dt, const void *o, ttt_dtype h_dt, const void *y,
                       ttt_dtype y_dt, const void *w, const void *gate, int gate_kind, const void *w_next,
                       ttt_dtype w_dt, float alpha, float beta, float eps, int64_t rows, int d, void *dh, void *dy,
                       float *dw, void *dgate, float *dw_next, void *ws, size_t ws_bytes, void *hip_stream) {
  static const char *kWhere = "ttt_norm_post_grad";
  const bool next = dx != nullptr;
  int rc = check_norm(kWhere, h_dt, y_dt, x_dt, w_dt, true, next, alpha, beta, eps, rows, d);
  if (!rc) rc = check_gate(kWhere, gate, gate_kind, rows);
  if (rc) return rc;
  const bool token = gate_kind == TTT_GATE_TOKEN;
  if (rows > 0 && (!dh_in && !dx)) return ttt_fail(TTT_E_NULL, "%s: dh_in and dx are both NULL", kWhere);
  if (rows > 0 && ((next && !o) || !y || !dh || !dy)) return ttt_fail(TTT_E_NULL, "%s: o, y, dh or dy is NULL", kWhere);
  if (rows > 0 && token && !dgate) return ttt_fail(TTT_E_NULL, "%s: dgate is NULL", kWhere);
  if (gate_kind == TTT_GATE_NONE) gate = dgate = nullptr;
  float *dgate_c = token ? nullptr : (float *)dgate;
  // without dx no gradient reaches w_next; in a call without rows dx says nothing, and dw_next is zero
  if (!next && rows > 0) dw_next = nullptr;
  const bool part = dw || dgate_c || dw_next;
  if (part && (rc = check_ws(kWhere, ws, ws_bytes, norm_ws_bytes(rows, d)))) return rc;
  const size_t n = (size_t)rows * d, hs = size_of(h_dt), ys = size_of(y_dt), ps = size_of(w_dt);
  rc = check_spans(kWhere,
                   {{"dh_in", dh_in, n * hs, hs},
                    {"dx", dx, n * size_of(x_dt), next ? size_of(x_dt) : 1},
                    {"o", next ? o : nullptr, n * hs, hs},
                    {"y", y, n * ys, ys},
                    {"w", w, d * ps, ps},
                    {"gate", gate, gate_bytes(gate_kind, rows, d, ys, ps), token ? ys : ps},
                    {"w_next", w_next, d * ps, ps}},
                   {{"dh", dh, n * hs, hs},
                    {"dy", dy, n * ys, ys},
                    {"dw", dw, (size_t)d * 4, 4},
                    {"dgate", dgate, gate_bytes(gate_kind, rows, d, ys, 4), token ? ys : 4},
                    {"dw_next", dw_next, (size_t)d * 4, 4},
                    {"ws", part ? ws : nullptr, norm_ws_bytes(rows, d), 4}},
                   {{dh, dh_in}, {dy, y}});
  if (rc) return rc;
  rc = ttt_check_device();
  if (rc) return rc;
  NormArgs a{};
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  a.alpha = alpha;
  a.beta = beta;
  a.h = o;
  a.y = y;
  a.w = w;
  a.gate = gate;
  a.token_gate = token;
  a.w_next = w_next;
  a.p_f32 = w_dt == TTT_F32;
  a.dx = dx;
  a.dh_in = dh_in;
  a.dh = dh;
  a.dy = dy;
  a.dgate_t = token ? dgate : nullptr;
  a.dw = dw;
  a.dgate_c = dgate_c;
  a.dw_next = dw_next;
  a.part = part ? (float *)ws : nullptr;
  return ttt_launched(launch_norm_bwd(a, types(h_dt, y_dt, x_dt), true, next, (hipStream_t)hip_stream), kWhere);
}

int ttt_embed(const void *E, ttt_dtype E_dt, int vocab, int d, const int32_t *ids, int64_t ids_ld, int B, int T,
              float scale, void *x, ttt_dtype x_dt, void *hip_stream) {
  static const char *kWhere = "ttt_embed";
  if (!known(E_dt) || !known(x_dt)) return ttt_fail(TTT_E_DTYPE, "%s: unknown dtype", kWhere);
  int rc = check_tokens(kWhere, B, T, ids_ld, vocab, d, scale);
  if (rc) return rc;
  const long long n = (long long)B * T;
  if (n > 0 && (!E || !ids || !x)) return ttt_fail(TTT_E_NULL, "%s: E, ids or x is NULL", kWhere);
  rc = check_spans(kWhere,
                   {{"E", E, (size_t)vocab * d * size_of(E_dt), size_of(E_dt)},
                    {"ids", ids, ids_bytes(B, T, ids_ld), 4}},
                   {{"x", x, (size_t)n * d * size_of(x_dt), size_of(x_dt)}}, {});
  if (rc) return rc;
  rc = ttt_check_device();
  if (rc) return rc;
  EmbedArgs a{};
  a.ids = TokenIds{ids, ids_ld, T, (int)n};
  a.E = E;
  a.x = x;
  a.vocab = vocab;
  a.d = d;
  a.scale = scale;
  return ttt_launched(launch_embed(a, E_dt == TTT_F32, x_dt == TTT_F32, (hipStream_t)hip_stream), kWhere);
}

int ttt_embed_grad_ws_bytes(int B, int T, int vocab, int d, size_t *bytes) {
  if (!bytes) return ttt_fail(TTT_E_NULL, "ttt_embed_grad_ws_bytes: bytes is NULL");
  const int rc = check_tokens("ttt_embed_grad_ws_bytes", B, T, T, vocab, d, 1.f);
  if (rc) return rc;
  *bytes = embed_grad_ws_bytes((long long)B * T, vocab, d);
  return TTT_OK;
}

int ttt_embed_grad(const void *dx, ttt_dtype dx_dt, const int32_t *ids, int64_t ids_ld, int B, int T, float scale,
                   int vocab, int d, void *dE, ttt_dtype dE_dt, int accumulate, void *ws, size_t ws_bytes,
                   void *hip_stream) {
  static const char *kWhere = "ttt_embed_grad";
  if (!known(dx_dt) || !known(dE_dt)) return ttt_fail(TTT_E_DTYPE, "%s: unknown dtype", kWhere);
  int rc = check_tokens(kWhere, B, T, ids_ld, vocab, d, scale);
  if (rc) return rc;
  const long long n = (long long)B * T;
  if (n > 0 && (!dx || !ids)) return ttt_fail(TTT_E_NULL, "%s: dx or ids is NULL", kWhere);
  if (!dE) return ttt_fail(TTT_E_NULL, "%s: dE is NULL", kWhere);
  const size_t need = embed_grad_ws_bytes(n, vocab, d);
  rc = check_ws(kWhere, ws, ws_bytes, need);
  if (rc) return rc;
  rc = check_spans(kWhere,
                   {{"dx", dx, (size_t)n * d * size_of(dx_dt), size_of(dx_dt)},
                    {"ids", ids, ids_bytes(B, T, ids_ld), 4}},
                   {{"dE", dE, (size_t)vocab * d * size_of(dE_dt), size_of(dE_dt)}, {"ws", ws, need, 4}}, {});
  if (rc) return rc;
  rc = ttt_check_device();
  if (rc) return rc;
  EmbedGradArgs a{};
  a.ids = TokenIds{ids, ids_ld, T, (int)n};
  a.dx = dx;
  a.dE = dE;
  a.vocab = vocab;
  a.d = d;
  a.accumulate = accumulate != 0;
  a.scale = scale;
  a.ws = ws;
  return ttt_launched(launch_embed_grad(a, dx_dt == TTT_F32, dE_dt == TTT_F32, (hipStream_t)hip_stream), kWhere);
}

int ttt_grad_ws_bytes(int n, size_t *bytes) {
  if (!bytes) return ttt_fail(TTT_E_NULL, "ttt_grad_ws_bytes: bytes is NULL");
  if (n < 0 || n > kMaxTensors) return ttt_fail(TTT_E_SHAPE, "ttt_grad_ws_bytes: n must be in [0, 2^20], got %d", n);
  *bytes = grad_ws(n);
  return TTT_OK;
}

int ttt_grad_norm(const void *const *grads, const int64_t *numel, const int32_t *dt, int n, float *norm, void *ws,
                  size_t ws_bytes, void *hip_stream) {
  static const char *kWhere = "ttt_grad_norm";
  try {
    int rc = check_grads(kWhere, grads, numel, dt, n, norm, ws, ws_bytes);
    if (rc) return rc;
    std::vector<Extent> e;
    for (int i = 0; i < n; ++i)
      if (numel[i])
        e.push_back({(uintptr_t)grads[i], (uintptr_t)grads[i] + numel[i] * size_of((ttt_dtype)dt[i]), false});
    e.push_back({(uintptr_t)norm, (uintptr_t)norm + 4, true});
    e.push_back({(uintptr_t)ws, (uintptr_t)ws + grad_ws(n), true});
    rc = check_extents(kWhere, e);
    if (!rc) rc = ttt_check_device();
    if (rc) return rc;
    return run_grads(kWhere, grad_tables(grads, numel, dt, n, nullptr), nullptr, 0.f, norm, ws,
                     (hipStream_t)hip_stream);
  } catch (...) {
    return ttt_fail(TTT_E_NOMEM, "%s: out of host memory", kWhere);
  }
}

int ttt_clip_grads(const void *const *grads, const int64_t *numel, const int32_t *dt, int n, float tau,
                   void *const *out, float *norm, void *ws, size_t ws_bytes, void *hip_stream) {
  static const char *kWhere = "ttt_clip_grads";
  try {
    int rc = check_grads(kWhere, grads, numel, dt, n, norm, ws, ws_bytes);
    if (rc) return rc;
    if (!(tau > 0.f)) return ttt_fail(TTT_E_ARG, "%s: tau must be greater than 0", kWhere);
    std::vector<Extent> e;
    for (int i = 0; i < n; ++i) {
      if (!numel[i]) continue;
      const size_t elem = size_of((ttt_dtype)dt[i]), bytes = numel[i] * elem;
      const void *o = out ? out[i] : grads[i];
      if (!o) return ttt_fail(TTT_E_NULL, "%s: output %d is NULL", kWhere, i);
      if ((uintptr_t)o % elem) return ttt_fail(TTT_E_ARG, "%s: output %d is not aligned to its elements", kWhere, i);
      e.push_back({(uintptr_t)o, (uintptr_t)o + bytes, true});
      if (o != grads[i]) e.push_back({(uintptr_t)grads[i], (uintptr_t)grads[i] + bytes, false});
    }
    e.push_back({(uintptr_t)norm, (uintptr_t)norm + 4, true});
    e.push_back({(uintptr_t)ws, (uintptr_t)ws + grad_ws(n), true});
    rc = check_extents(kWhere, e);
    if (!rc) rc = ttt_check_device();
    if (rc) return rc;
    const std::vector<GradTable> tables = grad_tables(grads, numel, dt, n, nullptr);
    if (!out) return run_grads(kWhere, tables, &tables, tau, norm, ws, (hipStream_t)hip_stream);
    const std::vector<GradTable> copies = grad_tables(grads, numel, dt, n, out);
    return run_grads(kWhere, tables, &copies, tau, norm, ws, (hipStream_t)hip_stream);
  } catch (...) {
    return ttt_fail(TTT_E_NOMEM, "%s: out of host memory", kWhere);
  }
}

}  // extern "C"

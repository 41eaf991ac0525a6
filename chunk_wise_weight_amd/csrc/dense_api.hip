// C ABI of the plain layers and of the AdamW step: argument checks and
// launches. No call allocates on the device, keeps state or waits.
#include <algorithm>
#include <cmath>
#include <vector>

#include "adamw.h"
#include "checks.h"
#include "linear.h"

namespace {

constexpr int kMaxDense = 1 << 20;  // widths

int check_dense(const char *where, ttt_dtype dt, int64_t rows, int in, int out) {
  if (!known(dt)) return ttt_fail(TTT_E_DTYPE, "%s: unknown dtype", where);
  if (rows < 0 || rows > kMaxRows)
    return ttt_fail(TTT_E_SHAPE, "%s: rows must be in [0, 2^31), got %lld", where, (long long)rows);
  if (in < 1 || in > kMaxDense || out < 1 || out > kMaxDense)
    return ttt_fail(TTT_E_SHAPE, "%s: widths must be in [1, 2^20], got %d and %d", where, in, out);
  return TTT_OK;
}

int check_y(const char *where, ttt_dtype dt, ttt_dtype y_dt) {
  if (!known(y_dt)) return ttt_fail(TTT_E_DTYPE, "%s: unknown dtype", where);
  if (dt == TTT_F32 && y_dt == TTT_BF16) return ttt_fail(TTT_E_DTYPE, "%s: fp32 products give an fp32 y", where);
  return TTT_OK;
}

int check_act(const char *where, int act, bool gated) {
  if (act < TTT_ACT_NONE || act > TTT_ACT_RELU || (gated && act == TTT_ACT_NONE))
    return ttt_fail(TTT_E_ARG, "%s: unknown activation %d", where, act);
  return TTT_OK;
}

// A workspace of `need` bytes; none is asked for where that is zero.
int check_scratch(const char *where, const void *ws, size_t have, size_t need) {
  return need ? check_ws(where, ws, have, need) : TTT_OK;
}

size_t padded(size_t bytes) { return (bytes + 15) / 16 * 16; }

GemmForm form(ttt_dtype dt, bool a_trans, bool b_trans, bool pair, bool out_f32) {
  GemmForm f;
  f.f32 = dt == TTT_F32;
  f.a_trans = a_trans;
  f.b_trans = b_trans;
  f.pair = pair;
  f.out_f32 = out_f32;
  return f;
}

// The products by their sizes: y[rows][out] = x W^T (pair: of both weights), dx[rows][in] = q W over one or two pairs,
// dW[out][in] = q^T x for one or two q.
GemmArgs sizes_y(int64_t rows, int in, int out) {
  GemmArgs g{};
  g.lda = g.ldb = g.nk = in;
  g.ni = g.ldo = out;
  g.nj = rows;
  g.segments = g.batch = 1;
  g.scale = 1.f;
  return g;
}
// ldq: from one row of q to the next
GemmArgs sizes_dx(int64_t rows, int in, int out, int pairs, int ldq) {
  GemmArgs g{};
  g.lda = g.ldo = g.ni = in;
  g.ldb = ldq;
  g.nk = out;
  g.nj = rows;
  g.segments = pairs;
  g.batch = 1;
  g.scale = 1.f;
  return g;
}
GemmArgs sizes_dw(int64_t rows, int in, int out, int count, int ldq) {
  GemmArgs g{};
  g.lda = g.ldo = g.ni = in;
  g.ldb = ldq;
  g.nj = out;
  g.nk = rows;
  g.segments = 1;
  g.batch = count;
  g.scale = 1.f;
  return g;
}
GemmForm form_y(ttt_dtype dt, bool pair, ttt_dtype y) { return form(dt, false, false, pair, y == TTT_F32); }
GemmForm form_dx(ttt_dtype dt) { return form(dt, true, false, false, dt == TTT_F32); }
GemmForm form_dw(ttt_dtype dt) { return form(dt, true, true, false, dt == TTT_F32); }

// Workspace of the gradients: q (or dg and du), the biases' sums, the products' splits. Rows of q that is made start on
// whole pieces of eight, zero behind their ends, as the products would otherwise copy them (gated gradients of 8192 x
// 2560 x 9721 in bf16: 2013 -> 1589 us; of 2000 x 512 x 1365 in fp32, which were not copied: 185 -> 157).
struct GradScratch {
  size_t q, part, gemm;
  int ldq;
  size_t bytes() const { return q + part + gemm; }
};
int made_ld(int out) { return (out + 7) / 8 * 8; }
// q: q (or dg and du) is made, not dy itself
GradScratch grad_scratch(int64_t rows, int in, int out, ttt_dtype dt, int count, bool q) {
  GradScratch s;
  s.ldq = q ? made_ld(out) : out;
  s.q = q ? padded((size_t)rows * s.ldq * size_of(dt)) * count : 0;
  s.part = padded(act_grad_ws_bytes(rows, out, count == 2));
  s.gemm = padded(std::max(gemm_ws_bytes(sizes_dx(rows, in, out, count, s.ldq), form_dx(dt)),
                           gemm_ws_bytes(sizes_dw(rows, in, out, count, s.ldq), form_dw(dt))));
  return s;
}

int run_dx(const char *where, const void *const *q, int ldq, const void *const *W, int pairs, ttt_dtype dt, float scale,
           int64_t rows, int in, int out, void *dx, void *ws, hipStream_t s) {
  GemmArgs g = sizes_dx(rows, in, out, pairs, ldq);
  for (int i = 0; i < pairs; ++i) {
    g.a[i] = W[i];
    g.b[i] = q[i];
  }
  g.out[0] = dx;
  g.scale = scale;
  g.ws = ws;
  return ttt_launched(launch_gemm(g, form_dx(dt), s), where);
}

int run_dw(const char *where, const void *const *q, int ldq, const void *x, int count, ttt_dtype dt, float scale,
           int64_t rows, int in, int out, void *const *dW, int accumulate, void *ws, hipStream_t s) {
  GemmArgs g = sizes_dw(rows, in, out, count, ldq);
  g.a[0] = x;
  for (int i = 0; i < count; ++i) {
    g.b[i] = q[i];
    g.out[i] = dW[i];
    g.res[i] = accumulate ? dW[i] : nullptr;
  }
  g.scale = scale;
  g.ws = ws;
  return ttt_launched(launch_gemm(g, form_dw(dt), s), where);
}

// ---- many tensors ----

constexpr int kMaxTensors = 1 << 20;
constexpr long long kMaxNumel = 1LL << 40;
constexpr long long kStreamAdam = 512LL << 20;  // arrays of more bytes pass by the caches

// Tables of the tensors that have elements. With `join`, tensors that follow
// one another in every array (views of flat buffers) are taken as one.
struct Many {
  void *const *w, *const *m, *const *v, *const *copies;
  const void *const *g;
  int16_t *const *tops;
  const int64_t *numel;
  const int32_t *w_dt, *g_dt;
  int n, state;  // bytes of a moment
};

size_t block_count(int64_t n) { return (size_t)((n + kAdamBlock - 1) / kAdamBlock); }

template <class Launch>
int run_many(const Many &a, bool join, Launch &&launch) {
  AdamTable t;
  long long last = 0;  // elements of the table's last tensor
  auto chunks = [](long long n) { return (uint32_t)((n + kAdamChunk - 1) / kAdamChunk); };
  auto close = [&](long long n) {
    t.first[t.n] = t.first[t.n - 1] + chunks(n);
    t.tail[t.n - 1] = (uint32_t)(n - (long long)(chunks(n) - 1) * kAdamChunk);
  };
  auto follows = [](const void *p, long long bytes, const void *q) { return (const char *)p + bytes == (const char *)q; };
  t.n = 0;
  t.first[0] = 0;
  for (int i = 0; i < a.n; ++i) {
    const long long n = a.numel[i];
    if (n == 0) continue;
    const uint8_t wf = a.w_dt ? a.w_dt[i] == TTT_F32 : 1, gf = a.g_dt ? a.g_dt[i] == TTT_F32 : 1;
    bf16_t *copy = a.copies ? (bf16_t *)a.copies[i] : nullptr;
    const int k = t.n - 1;
    if (join && k >= 0 && t.w_f32[k] == wf && t.g_f32[k] == gf && !t.copy[k] == !copy &&
        follows(t.w[k], last * (wf ? 4 : 2), a.w[i]) && follows(t.g[k], last * (gf ? 4 : 2), a.g[i]) &&
        follows(t.m[k], last * a.state, a.m[i]) && follows(t.v[k], last * a.state, a.v[i]) &&
        (!copy || follows(t.copy[k], last * 2, copy))) {
      last += n;
      close(last);
      continue;
    }
    // the tensors of a table keep the numbers that follow tensor0's: an empty one in between starts a new table
    if (t.n && (t.n == kAdamTable || (!join && t.tensor0 + t.n != i))) {
      const int rc = launch(t);
      if (rc) return rc;
      t.n = 0;
    }
    if (t.n == 0) t.tensor0 = i;
    t.w[t.n] = a.w[i];
    t.m[t.n] = a.m[i];
    t.v[t.n] = a.v ? a.v[i] : nullptr;
    t.g[t.n] = a.g ? a.g[i] : nullptr;
    t.copy[t.n] = copy;
    t.top[t.n] = a.tops ? a.tops[i] : nullptr;
    t.w_f32[t.n] = wf;
    t.g_f32[t.n] = gf;
    ++t.n;
    last = n;
    close(n);
  }
  return t.n ? launch(t) : TTT_OK;
}

// An array of a list: there where it has bytes, and aligned; its extent is noted.
int check_array(const char *where, const char *name, int i, const void *p, size_t bytes, size_t elem, bool out,
                std::vector<Extent> &e) {
  if (!bytes) return TTT_OK;
  if (!p) return ttt_fail(TTT_E_NULL, "%s: %s of tensor %d is NULL", where, name, i);
  if ((uintptr_t)p % elem) return ttt_fail(TTT_E_ARG, "%s: %s of tensor %d is not aligned to its elements", where, name, i);
  // views of one buffer in their order are one extent
  if (!e.empty() && e.back().hi == (uintptr_t)p && e.back().out == out)
    e.back().hi += bytes;
  else
    e.push_back({(uintptr_t)p, (uintptr_t)p + bytes, out});
  return TTT_OK;
}

int check_list(const char *where, const int64_t *numel, int n) {
  if (n < 0 || n > kMaxTensors) return ttt_fail(TTT_E_SHAPE, "%s: n must be in [0, 2^20], got %d", where, n);
  if (n > 0 && !numel) return ttt_fail(TTT_E_NULL, "%s: numel is NULL", where);
  long long total = 0;
  for (int i = 0; i < n; ++i)
    if (numel[i] < 0 || numel[i] > kMaxNumel || (total += numel[i]) > kMaxNumel)
      return ttt_fail(TTT_E_SHAPE, "%s: tensor %d has %lld elements; together at most 2^40 are taken", where, i,
                      (long long)numel[i]);
  return TTT_OK;
}

// one number on the device
int check_scalar(const char *where, const char *name, const void *p, size_t bytes, std::vector<Extent> &e) {
  if (!p) return TTT_OK;
  if ((uintptr_t)p % bytes) return ttt_fail(TTT_E_ARG, "%s: %s is not aligned to its elements", where, name);
  e.push_back({(uintptr_t)p, (uintptr_t)p + bytes, false});
  return TTT_OK;
}

}  // namespace

extern "C" {

int ttt_linear_ws_bytes(int64_t rows, int in, int out, ttt_dtype dt, size_t *bytes) {
  if (!bytes) return ttt_fail(TTT_E_NULL, "ttt_linear_ws_bytes: bytes is NULL");
  const int rc = check_dense("ttt_linear_ws_bytes", dt, rows, in, out);
  if (rc) return rc;
  *bytes = gemm_ws_bytes(sizes_y(rows, in, out), form_y(dt, false, dt));
  return TTT_OK;
}

int ttt_linear(const void *x, const void *W, ttt_dtype dt, const void *bias, int act, float scale,
               const void *residual, int64_t rows, int in, int out, void *pre, void *y, ttt_dtype y_dt, void *ws,
               size_t ws_bytes, void *hip_stream) {
  static const char *kWhere = "ttt_linear";
  int rc = check_dense(kWhere, dt, rows, in, out);
  if (!rc) rc = check_y(kWhere, dt, y_dt);
  if (!rc) rc = check_act(kWhere, act, false);
  if (rc) return rc;
  if (!std::isfinite(scale)) return ttt_fail(TTT_E_ARG, "%s: scale must be finite", kWhere);
  if (!W || (rows > 0 && (!x || !y))) return ttt_fail(TTT_E_NULL, "%s: x, W or y is NULL", kWhere);
  size_t need = 0;
  rc = ttt_linear_ws_bytes(rows, in, out, dt, &need);
  if (!rc) rc = check_scratch(kWhere, ws, ws_bytes, need);
  if (rc) return rc;
  const size_t e = size_of(dt), ye = size_of(y_dt), no = (size_t)rows * out;
  rc = check_spans(kWhere,
                   {{"x", x, (size_t)rows * in * e, e},
                    {"W", W, (size_t)out * in * e, e},
                    {"bias", bias, out * e, e},
                    {"residual", residual, no * ye, ye}},
                   {{"pre", pre, no * e, e}, {"y", y, no * ye, ye}, {"ws", need ? ws : nullptr, need, 4}},
                   {{y, residual}});
  if (!rc) rc = ttt_check_device();
  if (rc || rows == 0) return rc;
  GemmArgs g = sizes_y(rows, in, out);
  g.a[0] = W;
  g.b[0] = x;
  g.bias[0] = bias;
  g.res[0] = residual;
  g.pre[0] = pre;
  g.out[0] = y;
  g.scale = scale;
  g.act = act;
  g.ws = ws;
  return ttt_launched(launch_gemm(g, form_y(dt, false, y_dt), (hipStream_t)hip_stream), kWhere);
}

int ttt_gated_ws_bytes(int64_t rows, int in, int f, ttt_dtype dt, size_t *bytes) {
  if (!bytes) return ttt_fail(TTT_E_NULL, "ttt_gated_ws_bytes: bytes is NULL");
  const int rc = check_dense("ttt_gated_ws_bytes", dt, rows, in, f);
  if (rc) return rc;
  *bytes = gemm_ws_bytes(sizes_y(rows, in, f), form_y(dt, true, dt));
  return TTT_OK;
}

int ttt_gated(const void *x, const void *W_gate, const void *W_up, ttt_dtype dt, const void *b_gate, const void *b_up,
              int act, int64_t rows, int in, int f, void *g, void *u, void *z, void *ws, size_t ws_bytes,
              void *hip_stream) {
  static const char *kWhere = "ttt_gated";
  int rc = check_dense(kWhere, dt, rows, in, f);
  if (!rc) rc = check_act(kWhere, act, true);
  if (rc) return rc;
  if (!W_gate || !W_up || (rows > 0 && (!x || !z)))
    return ttt_fail(TTT_E_NULL, "%s: x, W_gate, W_up or z is NULL", kWhere);
  if (!b_gate != !b_up) return ttt_fail(TTT_E_NULL, "%s: one of b_gate, b_up is NULL", kWhere);
  if (rows > 0 && !g != !u) return ttt_fail(TTT_E_NULL, "%s: one of g, u is NULL", kWhere);
  size_t need = 0;
  rc = ttt_gated_ws_bytes(rows, in, f, dt, &need);
  if (!rc) rc = check_scratch(kWhere, ws, ws_bytes, need);
  if (rc) return rc;
  const size_t e = size_of(dt), nw = (size_t)f * in * e, no = (size_t)rows * f * e;
  rc = check_spans(kWhere,
                   {{"x", x, (size_t)rows * in * e, e},
                    {"W_gate", W_gate, nw, e},
                    {"W_up", W_up, nw, e},
                    {"b_gate", b_gate, f * e, e},
                    {"b_up", b_up, f * e, e}},
                   {{"g", g, no, e}, {"u", u, no, e}, {"z", z, no, e}, {"ws", need ? ws : nullptr, need, 4}}, {});
  if (!rc) rc = ttt_check_device();
  if (rc || rows == 0) return rc;
  GemmArgs a = sizes_y(rows, in, f);
  a.a[0] = W_gate;
  a.a[1] = W_up;
  a.b[0] = x;
  a.bias[0] = b_gate;
  a.bias[1] = b_up;
  a.pre[0] = g;
  a.pre[1] = u;
  a.out[0] = z;
  a.act = act;
  a.ws = ws;
  return ttt_launched(launch_gemm(a, form_y(dt, true, dt), (hipStream_t)hip_stream), kWhere);
}

int ttt_linear_grad_ws_bytes(int64_t rows, int in, int out, ttt_dtype dt, ttt_dtype y_dt, int act, size_t *bytes) {
  static const char *kWhere = "ttt_linear_grad_ws_bytes";
  if (!bytes) return ttt_fail(TTT_E_NULL, "%s: bytes is NULL", kWhere);
  int rc = check_dense(kWhere, dt, rows, in, out);
  if (!rc) rc = check_y(kWhere, dt, y_dt);
  if (!rc) rc = check_act(kWhere, act, false);
  if (rc) return rc;
  *bytes = grad_scratch(rows, in, out, dt, 1, act != TTT_ACT_NONE || y_dt != dt).bytes();
  return TTT_OK;
}

int ttt_linear_grad(const void *dy, ttt_dtype y_dt, const void *x, const void *W, ttt_dtype dt, const void *pre,
                    int act, float scale, int64_t rows, int in, int out, void *dx, void *dW, float *dbias,
                    int accumulate, void *ws, size_t ws_bytes, void *hip_stream) {
  static const char *kWhere = "ttt_linear_grad";
  int rc = check_dense(kWhere, dt, rows, in, out);
  if (!rc) rc = check_y(kWhere, dt, y_dt);
  if (!rc) rc = check_act(kWhere, act, false);
  if (rc) return rc;
  if (!std::isfinite(scale)) return ttt_fail(TTT_E_ARG, "%s: scale must be finite", kWhere);
  if (act == TTT_ACT_NONE) pre = nullptr;
  if (rows > 0 && (!dy || (dW && !x) || (dx && !W) || (act != TTT_ACT_NONE && !pre)))
    return ttt_fail(TTT_E_NULL, "%s: dy, x, W or pre is NULL", kWhere);
  // dy itself serves as q where it has the products' type; the scale is then theirs
  const bool made = act != TTT_ACT_NONE || y_dt != dt;
  const GradScratch sc = grad_scratch(rows, in, out, dt, 1, made);
  rc = check_ws(kWhere, ws, ws_bytes, sc.bytes());
  if (rc) return rc;
  const size_t e = size_of(dt), ye = size_of(y_dt), no = (size_t)rows * out, ni = (size_t)rows * in;
  const size_t nw = (size_t)out * in;
  rc = check_spans(kWhere,
                   {{"dy", dy, no * ye, ye}, {"x", x, ni * e, e}, {"W", W, nw * e, e}, {"pre", pre, no * e, e}},
                   {{"dx", dx, ni * e, e},
                    {"dW", dW, nw * e, e},
                    {"dbias", dbias, (size_t)out * 4, 4},
                    {"ws", ws, sc.bytes(), 4}},
                   {});
  if (!rc) rc = ttt_check_device();
  if (rc) return rc;
  const hipStream_t s = (hipStream_t)hip_stream;
  const bool pass = rows > 0 && made;
  const void *q = pass ? ws : dy;
  if (pass || dbias) {
    ActGradArgs a{};
    a.dy = dy;
    a.p = pre;
    a.out = pass ? ws : nullptr;
    a.sum = dbias;
    a.part = (float *)((char *)ws + sc.q);
    a.rows = rows;
    a.n = out;
    a.ldo = sc.ldq;
    a.scale = scale;
    a.act = act;
    a.accumulate = accumulate != 0;
    a.dy_f32 = y_dt == TTT_F32;
    a.f32 = dt == TTT_F32;
    rc = ttt_launched(launch_act_grad(a, s), kWhere);
    if (rc) return rc;
  }
  const float left = pass ? 1.f : scale;
  void *split_ws = (char *)ws + sc.q + sc.part;
  if (dx && rows > 0) rc = run_dx(kWhere, &q, sc.ldq, &W, 1, dt, left, rows, in, out, dx, split_ws, s);
  if (dW && !rc) rc = run_dw(kWhere, &q, sc.ldq, x, 1, dt, left, rows, in, out, &dW, accumulate, split_ws, s);
  return rc;
}

int ttt_gated_grad_ws_bytes(int64_t rows, int in, int f, ttt_dtype dt, size_t *bytes) {
  if (!bytes) return ttt_fail(TTT_E_NULL, "ttt_gated_grad_ws_bytes: bytes is NULL");
  const int rc = check_dense("ttt_gated_grad_ws_bytes", dt, rows, in, f);
  if (rc) return rc;
  *bytes = grad_scratch(rows, in, f, dt, 2, true).bytes();
  return TTT_OK;
}

int ttt_gated_grad(const void *dz, const void *x, const void *W_gate, const void *W_up, ttt_dtype dt, const void *g,
                   const void *u, int act, int64_t rows, int in, int f, void *dx, void *dW_gate, void *dW_up,
                   float *db_gate, float *db_up, int accumulate, void *ws, size_t ws_bytes, void *hip_stream) {
  static const char *kWhere = "ttt_gated_grad";
  int rc = check_dense(kWhere, dt, rows, in, f);
  if (!rc) rc = check_act(kWhere, act, true);
  if (rc) return rc;
  if (!dW_gate != !dW_up || !db_gate != !db_up)
    return ttt_fail(TTT_E_NULL, "%s: one of dW_gate, dW_up or of db_gate, db_up is NULL", kWhere);
  if (rows > 0 && (!dz || !g || !u || (dW_gate && !x) || (dx && (!W_gate || !W_up))))
    return ttt_fail(TTT_E_NULL, "%s: dz, x, W_gate, W_up, g or u is NULL", kWhere);
  const GradScratch sc = grad_scratch(rows, in, f, dt, 2, true);
  rc = check_ws(kWhere, ws, ws_bytes, sc.bytes());
  if (rc) return rc;
  const size_t e = size_of(dt), no = (size_t)rows * f * e, ni = (size_t)rows * in * e, nw = (size_t)f * in * e;
  rc = check_spans(kWhere,
                   {{"dz", dz, no, e}, {"x", x, ni, e}, {"W_gate", W_gate, nw, e}, {"W_up", W_up, nw, e},
                    {"g", g, no, e}, {"u", u, no, e}},
                   {{"dx", dx, ni, e},
                    {"dW_gate", dW_gate, nw, e},
                    {"dW_up", dW_up, nw, e},
                    {"db_gate", db_gate, (size_t)f * 4, 4},
                    {"db_up", db_up, (size_t)f * 4, 4},
                    {"ws", ws, sc.bytes(), 4}},
                   {});
  if (!rc) rc = ttt_check_device();
  if (rc) return rc;
  const hipStream_t s = (hipStream_t)hip_stream;
  const void *q[2] = {ws, (char *)ws + sc.q / 2}, *W[2] = {W_gate, W_up};
  void *dW[2] = {dW_gate, dW_up};
  if (rows > 0 || db_gate) {
    ActGradArgs a{};
    a.dy = dz;
    a.p = g;
    a.u = u ? u : (const void *)ws;  // without rows nothing of it is read
    a.out = (void *)q[0];
    a.out2 = (void *)q[1];
    a.sum = db_gate;
    a.sum2 = db_up;
    a.part = (float *)((char *)ws + sc.q);
    a.rows = rows;
    a.n = f;
    a.ldo = sc.ldq;
    a.scale = 1.f;
    a.act = act;
    a.accumulate = accumulate != 0;
    a.dy_f32 = a.f32 = dt == TTT_F32;
    rc = ttt_launched(launch_act_grad(a, s), kWhere);
    if (rc) return rc;
  }
  void *split_ws = (char *)ws + sc.q + sc.part;
  if (dx && rows > 0) rc = run_dx(kWhere, q, sc.ldq, W, 2, dt, 1.f, rows, in, f, dx, split_ws, s);
  if (dW_gate && !rc) rc = run_dw(kWhere, q, sc.ldq, x, 2, dt, 1.f, rows, in, f, dW, accumulate, split_ws, s);
  return rc;
}

int ttt_dense_plan(int product, int64_t rows, int in, int out, ttt_dtype dt, int q_made, int *kernel, int *tile,
                   int *splits, int *copies) {
  static const char *kWhere = "ttt_dense_plan";
  const int rc = check_dense(kWhere, dt, rows, in, out);
  if (rc) return rc;
  const bool gated = product == TTT_PRODUCT_GATED_DX || product == TTT_PRODUCT_GATED_DW;
  const int ldq = gated || q_made ? made_ld(out) : out;
  GemmPlan p{};
  switch (product) {
    case TTT_PRODUCT_LINEAR: p = gemm_plan(sizes_y(rows, in, out), form_y(dt, false, dt)); break;
    case TTT_PRODUCT_GATED: p = gemm_plan(sizes_y(rows, in, out), form_y(dt, true, dt)); break;
    case TTT_PRODUCT_LINEAR_DX:
    case TTT_PRODUCT_GATED_DX: p = gemm_plan(sizes_dx(rows, in, out, gated ? 2 : 1, ldq), form_dx(dt)); break;
    case TTT_PRODUCT_LINEAR_DW:
    case TTT_PRODUCT_GATED_DW: p = gemm_plan(sizes_dw(rows, in, out, gated ? 2 : 1, ldq), form_dw(dt)); break;
    default: return ttt_fail(TTT_E_ARG, "%s: unknown product %d", kWhere, product);
  }
  if (kernel) *kernel = p.kernel;
  if (tile) *tile = p.tile;
  if (splits) *splits = p.splits;
  if (copies) *copies = p.copies;
  return TTT_OK;
}

int ttt_adamw(void *const *w, const int32_t *w_dt, const void *const *g, const int32_t *g_dt, void *const *m,
              void *const *v, int state_bits, int16_t *const *tops, void *const *copies, const int64_t *numel, int n,
              int64_t step, const int64_t *step_dev, double lr, const float *lr_dev, double beta1, double beta2,
              double eps, double weight_decay, const float *norm, double tau, uint32_t seed, void *hip_stream) {
  static const char *kWhere = "ttt_adamw";
  try {
    int rc = check_list(kWhere, numel, n);
    if (rc) return rc;
    if (state_bits != 8 && state_bits != 32)
      return ttt_fail(TTT_E_ARG, "%s: state_bits must be 8 or 32, got %d", kWhere, state_bits);
    const bool bits8 = state_bits == 8;
    if (n > 0 && (!w || !w_dt || !g || !g_dt || !m || !v || (bits8 && !tops)))
      return ttt_fail(TTT_E_NULL, "%s: a list is NULL", kWhere);
    if (!step_dev && step < 1) return ttt_fail(TTT_E_ARG, "%s: step must be at least 1, got %lld", kWhere, (long long)step);
    if (!(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1))
      return ttt_fail(TTT_E_ARG, "%s: beta1 and beta2 must be in [0, 1)", kWhere);
    if (!(eps >= 0) || !(weight_decay >= 0) || !std::isfinite(eps) || !std::isfinite(weight_decay) ||
        (!lr_dev && !std::isfinite(lr)))
      return ttt_fail(TTT_E_ARG, "%s: lr, eps and weight_decay must be finite, eps and weight_decay not negative", kWhere);
    if (norm && !(tau > 0)) return ttt_fail(TTT_E_ARG, "%s: tau must be greater than 0", kWhere);
    std::vector<Extent> ex;
    const size_t state = bits8 ? 1 : 4;
    for (int i = 0; i < n; ++i)
      if (!known((ttt_dtype)w_dt[i]) || !known((ttt_dtype)g_dt[i]))
        return ttt_fail(TTT_E_DTYPE, "%s: tensor %d has an unknown dtype", kWhere, i);
    auto list = [&](const char *name, const void *const *p, const int32_t *dt, size_t elem, bool out) {
      for (int i = 0; i < n && !rc; ++i) {
        const size_t size = dt ? size_of((ttt_dtype)dt[i]) : elem;
        rc = check_array(kWhere, name, i, p[i], (size_t)numel[i] * size, size, out, ex);
      }
    };
    list("w", w, w_dt, 0, true);
    list("g", g, g_dt, 0, false);
    list("m", m, nullptr, state, true);
    list("v", v, nullptr, state, true);
    for (int i = 0; i < n && !rc && bits8; ++i)
      rc = check_array(kWhere, "tops", i, tops[i], block_count(numel[i]) * 4, 2, true, ex);
    for (int i = 0; i < n && !rc && copies; ++i)
      if (copies[i]) rc = check_array(kWhere, "the copy", i, copies[i], (size_t)numel[i] * 2, 2, true, ex);
    if (!rc) rc = check_scalar(kWhere, "step_dev", step_dev, 8, ex);
    if (!rc) rc = check_scalar(kWhere, "lr_dev", lr_dev, 4, ex);
    if (!rc) rc = check_scalar(kWhere, "norm", norm, 4, ex);
    if (!rc) rc = check_extents(kWhere, ex);
    if (!rc) rc = ttt_check_device();
    if (rc) return rc;
    AdamArgs a{};
    a.decay1 = adam_decay(beta1);
    a.decay2 = adam_decay(beta2);
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.eps = eps > 0 ? std::max((float)eps, 0x1p-149f) : 0.f;  // an eps above 0 stays so: 0 / eps is 0
    a.lr = lr;
    a.decay = weight_decay;
    a.tau = tau;
    a.log1 = std::log(beta1);
    a.log2 = std::log(beta2);
    a.step = step;
    a.step_dev = (const long long *)step_dev;
    a.lr_dev = lr_dev;
    a.norm = norm;
    a.seed = seed;
    a.fixed.lr1 = (float)(lr / -std::expm1((double)step * a.log1));
    a.fixed.root2 = (float)(1.0 / std::sqrt(-std::expm1((double)step * a.log2)));
    a.fixed.shrink = (float)(lr * weight_decay);
    a.fixed.key = adam_key(seed, step);
    long long bytes = 0;
    for (const Extent &x : ex) bytes += (long long)(x.hi - x.lo);
    const bool stream = bytes > kStreamAdam;
    const Many all{w, m, v, copies, g, bits8 ? tops : nullptr, numel, w_dt, g_dt, n, (int)state};
    return run_many(all, !bits8, [&](const AdamTable &t) {
      return ttt_launched(launch_adamw(t, a, bits8, stream, (hipStream_t)hip_stream), kWhere);
    });
  } catch (...) {
    return ttt_fail(TTT_E_NOMEM, "%s: out of host memory", kWhere);
  }
}

int ttt_adamw_values(const void *const *codes, const int16_t *const *tops, int moment, float *const *out,
                     const int64_t *numel, int n, void *hip_stream) {
  static const char *kWhere = "ttt_adamw_values";
  try {
    int rc = check_list(kWhere, numel, n);
    if (rc) return rc;
    if (moment != 1 && moment != 2) return ttt_fail(TTT_E_ARG, "%s: moment must be 1 or 2, got %d", kWhere, moment);
    if (n > 0 && (!codes || !tops || !out)) return ttt_fail(TTT_E_NULL, "%s: a list is NULL", kWhere);
    std::vector<Extent> ex;
    for (int i = 0; i < n && !rc; ++i) {
      const size_t k = (size_t)numel[i];
      rc = check_array(kWhere, "codes", i, codes[i], k, 1, false, ex);
      if (!rc) rc = check_array(kWhere, "tops", i, tops[i], block_count(numel[i]) * 4, 2, false, ex);
      if (!rc) rc = check_array(kWhere, "out", i, out[i], k * 4, 4, true, ex);
    }
    if (!rc) rc = check_extents(kWhere, ex);
    if (!rc) rc = ttt_check_device();
    if (rc) return rc;
    long long bytes = 0;
    for (const Extent &x : ex) bytes += (long long)(x.hi - x.lo);
    const Many all{(void *const *)out, (void *const *)codes, nullptr, nullptr, nullptr, (int16_t *const *)tops,
                   numel, nullptr, nullptr, n, 1};
    return run_many(all, false, [&](const AdamTable &t) {
      return ttt_launched(launch_adamw_values(t, moment == 2, bytes > kStreamAdam, (hipStream_t)hip_stream), kWhere);
    });
  } catch (...) {
    return ttt_fail(TTT_E_NOMEM, "%s: out of host memory", kWhere);
  }
}

}  // extern "C"

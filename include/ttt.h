/*
 * ttt.h — C ABI of the MI355X (gfx950) chunk-wise fast-weight library.
 *
 * The library runs the hot path of In-Place Test-Time Training for one gated
 * MLP layer whose final projection W_down is the fast weight (paperlayer.ai
 * summary, sec. 3 "In-Place Adaptation"; iplexlaw.co.kr walkthrough, sec. 2):
 *
 *   Z        = SiLU(x W_gate^T) * (x W_up^T)          (W_up, W_gate frozen)
 *   V[t]     = E_tgt[ids[t+1]]                         (next-token target row)
 *   chunk i  : y[chunk i] = Z[chunk i] W_{i-1}^T       (apply, pre-update state)
 *              W_i = W_{i-1} + eta V[chunk i]^T Z[chunk i]   (update)
 *
 * The update rule is the pages' simplified form dW_down = eta V^T Z
 * (iplexlaw sec. 2 and sec. 4); apply-then-update over non-overlapping chunks
 * follows iplexlaw sec. 3 and paperlayer sec. 3 "Chunk-Wise Updates"; the
 * target is V^ = Conv1D(X0) W_target with the kernel reduced to the next-token
 * tap and W_target folded into E_tgt (paperlayer sec. 3 "LM-Aligned
 * Objective"); state reset at document ends follows paperlayer App. B.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers on the current HIP device,
 *     row-major, densely packed, owned by the caller. They must stay valid
 *     until the work queued on `hip_stream` has completed.
 *   - `hip_stream` is a hipStream_t (NULL = the default stream). Work is
 *     queued asynchronously; no call synchronises the host except where noted.
 *   - Argument errors are detected before any device work is queued.
 *   - Return value 0 = success; a negative TTT_E_* code otherwise, with a
 *     message available from ttt_last_error() (thread-local).
 *   - No C++ exception crosses the ABI. A handle is not thread-safe: calls on
 *     one handle must come from one thread at a time and, when they are on
 *     different streams, be ordered by the caller.
 *   - Only gfx950 devices are accepted (TTT_E_NODEV otherwise).
 */
#ifndef TTT_H
#define TTT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ttt_handle ttt_handle; /* opaque, owned by the library */

/* Activation/weight element type. The fast-weight state is always fp32.
 * The handle keeps each sequence's fast weight as D = W - W_down0, the change
 * since its last reset, in fp32 (W_down0 is kept beside it): the updates are
 * small next to W, and held this way they accumulate with fp32 relative
 * precision even when each one is far below the fp32 resolution of W itself
 * (as with clipped updates), also across calls.
 * TTT_F32:  x, W_up, W_gate, W_down0, E_tgt and y are float.
 * TTT_BF16: they are bfloat16 (uint16 bit patterns); matrix products run on
 *           bf16 MFMA with fp32 accumulation. */
typedef enum { TTT_F32 = 0, TTT_BF16 = 1 } ttt_dtype;

enum {
  TTT_OK = 0,
  TTT_E_NULL = -1,  /* a required pointer is NULL                           */
  TTT_E_SHAPE = -2, /* a size is out of range or violates an alignment rule */
  TTT_E_DTYPE = -3, /* unknown dtype                                         */
  TTT_E_NOMEM = -4, /* device allocation failed                              */
  TTT_E_HIP = -5,   /* a HIP runtime call or kernel launch failed            */
  TTT_E_NODEV = -6, /* no device, or the current device is not gfx950        */
  TTT_E_ARG = -7    /* other invalid argument (e.g. batch index, non-finite eta) */
};

/*
 * ttt_init — create a handle for one layer.
 *
 *   W_up, W_gate : [f][d] frozen up and gate projections (dtype `dt`).
 *   W_down0      : [d][f] initial fast weight (dtype `dt`). The three
 *                  weight pointers must be 16-byte aligned.
 *   d, f         : model width and hidden width, at most 65536; multiples of
 *                  64 on the fp32 path and of 256 on the bf16 path (the MFMA
 *                  kernels work on whole 256 x 256 tiles of the state).
 *   C            : chunk length in tokens, C >= 1. Chunks are counted from the
 *                  first token of each ttt_forward_chunked call.
 *   eta          : learning rate of the update (finite).
 *   max_batch    : number of independent sequences (fast-weight states) the
 *                  handle holds, 1 .. 4096.
 *
 * The library copies the weights into buffers it owns (re-laid out for its
 * kernels) and keeps an fp32 image of W_down0. Every state starts equal to
 * W_down0. The caller may free its weight buffers once the queued copies have
 * completed on `hip_stream`. On success *out receives the handle; on failure
 * *out is set to NULL and nothing is leaked.
 */
int ttt_init(ttt_handle **out, const void *W_up, const void *W_gate, const void *W_down0, int d, int f,
             int C, float eta, ttt_dtype dt, int max_batch, void *hip_stream);

/*
 * ttt_forward_chunked — run the chunk-wise apply-then-update scan over one
 * block of tokens for sequences 0 .. B-1.
 *
 *   x       : [B][T][d] layer input (dtype of the handle).
 *   ids     : [B][T+1] int32 token ids; ids[b][t] is the token at position t
 *             and ids[b][T] the look-ahead token after the block. The target
 *             of position t is row ids[b][t+1] of E_tgt; an id outside
 *             [0, vocab) (e.g. -1 at a document end) gives a zero target row.
 *   E_tgt   : [vocab][d] target-embedding table (dtype of the handle).
 *   B       : 0 .. max_batch. T: tokens per sequence, 0 .. 2^23.
 *   y       : [B][T][d] output (dtype of the handle), written in full.
 *   W_final : optional [B][d][f] fp32 output; receives each sequence's fast
 *             weight after the block, W_down0 + D rounded to fp32 (NULL = not
 *             wanted). ttt_state_delta gives D itself.
 *
 * x, E_tgt and y must be 16-byte aligned (TTT_E_ARG otherwise).
 *
 * Each sequence starts from its current state (W_down0 after init or reset,
 * else what the previous call left) and keeps the final state in the handle,
 * so consecutive calls continue one stream (the last chunk of a call may be
 * short; to continue chunking seamlessly, make T a multiple of C). Scratch
 * memory is allocated by the library on first use and grown when B*T grows;
 * that allocation is the only point where this call may block the host.
 */
int ttt_forward_chunked(ttt_handle *h, const void *x, const int32_t *ids, const void *E_tgt, int vocab, int B,
                        int T, void *y, float *W_final, void *hip_stream);

/*
 * ttt_forward_chunked_noalloc — ttt_forward_chunked for callers that cannot
 * allocate device memory during the call: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc. Same arguments,
 * layouts, semantics and results (bit for bit) as ttt_forward_chunked, but the
 * scratch of the call (target rows, Z, snapshots, group scores,
 * clipping partials) lives in a fixed workspace of
 * TTT_NOALLOC_WORKSPACE_BYTES inside the library: a file-scope device array
 * that each GPU the library runs on holds until the process ends, its address
 * taken in ttt_init. The call performs no hipMalloc, hipFree or other
 * allocation. A call whose scratch would exceed the workspace returns
 * TTT_E_SHAPE before any device work, naming the bytes it needs (roughly
 * B*T*(4f + 2d) bytes plus 2*d*f per group of the plan on the bf16 path, so
 * small layers and short blocks; larger calls use ttt_forward_chunked).
 * Every call on one GPU shares that GPU's workspace, whichever handle it
 * comes from, and leaves its contents behind (each call writes every part it
 * reads): calls that overlap in time on one GPU, e.g. on two streams, race
 * and must be ordered by the caller.
 */
#define TTT_NOALLOC_WORKSPACE_BYTES ((size_t)64 << 20)
int ttt_forward_chunked_noalloc(ttt_handle *h, const void *x, const int32_t *ids, const void *E_tgt, int vocab,
                                int B, int T, void *y, float *W_final, void *hip_stream);

/*
 * ttt_forward_docs — ttt_forward_chunked over streams that pack several
 * documents (paperlayer App. B; iplexlaw sec. 6: the fast weight returns to its
 * initial value at document boundaries, so no state crosses between
 * independent documents).
 *   doc_counts : host array [B]; doc_counts[b] documents start inside
 *                sequence b's block besides the one it opens with (0 .. T-1).
 *   doc_starts : host array, the concatenated start positions: sequence b's
 *                are the next doc_counts[b] entries, strictly increasing inside
 *                (0, T). NULL allowed when every count is 0.
 * The first document continues the sequence's current state (like
 * ttt_forward_chunked); at every listed start the state returns to W_down0 and
 * chunking restarts from that token. A document's last target row lies in its
 * last chunk, whose update the reset discards, so no target crosses a
 * document end. The final state is the last document's, kept in the handle as
 * usual. On a bf16 handle with eta != 0 (also with clipping and the general
 * target) the call is one launch sequence in which every document is a
 * sequence of its own, with its own scratch slots and snapshot groups, and
 * the state a sequence's last document leaves is copied back once at the end.
 * On an fp32 handle, or with eta = 0, documents run one after the other on
 * the stream (B = 1 launches per document). With profiling on,
 * ttt_phase_times sums a call's launch sequences.
 * Other arguments, ownership and errors as ttt_forward_chunked.
 */
int ttt_forward_docs(ttt_handle *h, const void *x, const int32_t *ids, const void *E_tgt, int vocab, int B, int T,
                     const int32_t *doc_starts, const int32_t *doc_counts, void *y, float *W_final,
                     void *hip_stream);

/*
 * ttt_reset — restore the fast weight of sequence b (or of every sequence if
 * b == -1) to W_down0 (D = 0): the document-boundary reset (paperlayer App. B;
 * iplexlaw sec. 6). Queued on `hip_stream`.
 */
int ttt_reset(ttt_handle *h, int b, void *hip_stream);

/* ttt_destroy — free the handle and everything it owns (synchronises the device). NULL is a no-op. */
void ttt_destroy(ttt_handle *h);

/* ttt_last_error — message for the last nonzero return on this thread ("" if none). */
const char *ttt_last_error(void);

/*
 * ttt_set_group_chunks — tuning knob of the two-level scan (no effect on the
 * result beyond rounding). The library keeps each state resident across the
 * whole block of tokens and takes a snapshot of it (bf16 on the bf16 path,
 * fp32 on the fp32 path) at the start of every group of G chunks; the outputs
 * of a group are formed from its snapshot plus the block-causal term of the
 * earlier chunks inside the group. This is the pages' exclusive prefix over
 * chunk updates (iplexlaw sec. 6; paperlayer App. B) taken at two levels.
 * G = 0 restores the default (about 1024 tokens per group, rounded so that
 * G*C is a multiple of 64). G*C must be a multiple of 64; TTT_E_SHAPE
 * otherwise.
 */
int ttt_set_group_chunks(ttt_handle *h, int G);

/*
 * ttt_plan — host-only query of the layout a call with T tokens and chunk C
 * would use (no device work; usable without a GPU):
 *   *G       : chunks per snapshot group;  *L = G*C tokens per group;
 *   *ngroups : groups in the call (ceil(T / L));
 *   *T_pad   : token slots per sequence in the scratch buffers (T rounded up to 256).
 * When C >= T the call is a single chunk and C is taken as T.
 * Any output pointer may be NULL. `G_override` as in ttt_set_group_chunks.
 */
int ttt_plan(int T, int C, int G_override, int *G, int *L, int *ngroups, int *T_pad);

/*
 * ttt_set_target_conv — the general LM-aligned target V^ = Conv1D(X0) W_target
 * (paperlayer sec. 3 "LM-Aligned Objective"; iplexlaw sec. 4 and sec. 6, a
 * depthwise kernel of size 5 over the token embeddings and a learnable
 * projection) in place of the next-token rows of E_tgt.
 *   conv_w   : [K][d] depthwise tap weights (dtype of the handle); tap k of
 *              target row t reads the embedding of the token at position
 *              t+1+k (ids[b][t+1+k]).
 *   K        : 1 .. 64 taps; K = 0 restores the next-token target (the other
 *              arguments are then ignored).
 *   W_target : [d][d] projection (dtype of the handle): V^[t] = U[t] W_target.
 * After this call the E_tgt argument of ttt_forward_chunked is the token
 * embedding table X0 [vocab][d]. The chunk boundary pads the convolution: row t
 * of chunk i uses tap positions only up to min((i+1)C, T), the first token of
 * the next chunk (already that chunk's input); later taps are zero, so no output
 * depends on a later token. With K = 1, conv_w = 1 and W_target = I the result
 * equals the next-token target. Both arrays are copied (the caller may free
 * them once the stream has run the copy); they must be 16-byte aligned.
 * Synchronises `hip_stream`. Adds [B][T][d] of scratch per forward.
 */
int ttt_set_target_conv(ttt_handle *h, const void *conv_w, int K, const void *W_target, void *hip_stream);

/*
 * ttt_set_clip — Frobenius-norm clipping of each chunk update (paperlayer
 * App. C.2 "Inference Stability", threshold 1e-5 in the reported long-context
 * evaluations; iplexlaw sec. 6): with tau > 0, chunk i's update
 * dW_i = eta V_i^T Z_i is applied as dW_i * min(1, tau / ||dW_i||_F), in the
 * state and in the outputs of later chunks alike. tau = 0 or +inf turns it
 * off (the default); tau < 0 or NaN returns TTT_E_ARG. The norm is taken from
 * the chunk Grams, ||V_i^T Z_i||_F^2 = sum_{s,t in chunk i} <v_s,v_t><z_s,z_t>,
 * in fp32. Applies to later ttt_forward_chunked calls; needs extra scratch:
 * small fp32 buffers; on a bf16 handle 1 KB per token slot and per 256-token
 * span of a chunk (the Gram kernel's fp32 partial products: 128 MB at
 * T = 131072, C = 256); plus [B][T][d] target rows in the handle's dtype on
 * an fp32 handle or with the general target (a bf16 handle with the plain
 * target reads the rows from E_tgt through the ids when vocab*d*2 < 2^31).
 */
int ttt_set_clip(ttt_handle *h, float tau);

/*
 * ttt_state_delta — copy D = W - W_down0 of sequences 0 .. B-1, the change of
 * each fast weight since its last reset (or init), to dW ([B][d][f] fp32,
 * device, 16-byte aligned), queued on `hip_stream` after the work already
 * there. Where the updates are much smaller than W (clipped updates at the
 * pages' tau = 1e-5 move each element by about 1e-9 against |W| ~ 1e-2), the
 * fp32 W_final cannot resolve them (its rounding alone is about 3% of D
 * there), while D carries them at fp32 relative precision. B in [0,
 * max_batch] (TTT_E_SHAPE otherwise); dW NULL with B > 0 is TTT_E_NULL.
 */
int ttt_state_delta(ttt_handle *h, float *dW, int B, void *hip_stream);

/*
 * ttt_set_output_f32 — on a bf16 handle, later forward calls write y as fp32
 * ([B][T][d] float, 4 bytes per element) instead of bf16: the output GEMM's
 * fp32 accumulators are stored without the final rounding to bf16. The
 * fast-weight contribution to y is often a small fraction of y (a few percent
 * on short streams), and bf16 rounding of y alone then blurs it by up to
 * 2^-9 |y|; callers that keep a residual stream in fp32 avoid that rounding.
 * on = 0 restores bf16 y. No effect on an fp32 handle (y is always fp32).
 * Returns TTT_E_NULL for a NULL handle.
 */
int ttt_set_output_f32(ttt_handle *h, int on);

/*
 * ttt_set_profiling / ttt_phase_times — per-phase device timing of the
 * forward calls, from HIP events recorded on their streams.
 * Phases: 0 target gather, 1 up/gate GEMM + SwiGLU, 2 clipping factors
 * (0 when clipping is off), 3 state update with snapshots, 4 within-group
 * scores, 5 output GEMM, 6 final-state copy. With clipping on a bf16 handle
 * and the plain target, the gather runs after the factors (it applies them)
 * and counts in phase 2.
 * Each launch sequence (a ttt_forward_chunked call, or one document of a
 * ttt_forward_docs call) records one set of events in a ring of 16 sets, so
 * calls need not wait for each other. ttt_phase_times waits for the sets
 * recorded since the previous read and writes `n` (<= 7) milliseconds per
 * phase to ms[]: the sum over those sets divided by the number of forward
 * calls among them (the mean per call; a call with documents sums them).
 * With no call since the previous read it writes the previous figures again.
 * A phase that did not run reads only the spacing of its two events (a few
 * microseconds). When a launch sequence finds all 16 sets unread, the oldest
 * is folded into running sums first (the host waits for that set, recorded
 * 16 sequences earlier, to complete), so any number of calls or documents
 * may come between two reads. ttt_set_profiling resets the window.
 */
int ttt_set_profiling(ttt_handle *h, int on);
int ttt_phase_times(ttt_handle *h, float *ms, int n);

/* ttt_workspace_bytes — device bytes the handle currently owns (weights, states, scratch). */
int ttt_workspace_bytes(ttt_handle *h, size_t *bytes);

/*
 * What stands around the layers of a stack. These entry points take no
 * handle: each works on the arrays it is given, on the current device, and
 * keeps nothing between calls. They allocate nothing (where scratch is needed
 * the caller brings it, `ws`, 16-byte aligned, of at least the bytes the
 * matching _ws_bytes query names; its contents need not be kept, and calls
 * that may overlap in time need a workspace each), so they can be captured
 * into a HIP graph. Arrays need only the alignment of their elements. Unless
 * said otherwise an output may not overlap an input or another output
 * (TTT_E_ARG); where "in place" is allowed it means the very same array.
 */

/*
 * The norms around a block (rows of d elements, 8 <= d <= 65536):
 *
 *   rms(v)         = (mean(v^2) + eps)^-1/2 over the row
 *   ttt_norm_pre   : x = w * h * rms(h)                 the norm before a block
 *   ttt_norm_post  : o = alpha * h + beta * gate * w * y * rms(y)
 *                    the norm after a block, its gate and the residual scales;
 *                    with x not NULL also the next block's norm,
 *                    x = w_next * o * rms(o), of o before it is rounded
 *
 * With w = NULL the rows are normalised without a gain (the layer's
 * RMS-normalised input rows). Sums are fp32, and each result is rounded once:
 * |elements| of h, y and o past 1e18, whose squares leave fp32, are not
 * supported (a row's sum of squares may leave it).
 *
 *   rows    : 0 .. 2^31-1.
 *   h, o    : [rows][d] residual stream, h_dt. o may be h (in place).
 *   y       : [rows][d] what the block gave, y_dt.
 *   x       : [rows][d] the block's input, x_dt.
 *   types   : (h, x) fp32/fp32, fp32/bf16 or bf16/bf16; (h, y) the same three,
 *             or fp32/fp32 with a bf16 x.
 *   w, w_next : [d] gains, w_dt, or NULL (ones).
 *   gate    : TTT_GATE_NONE (gate ignored), TTT_GATE_CHANNEL ([d], w_dt) or
 *             TTT_GATE_TOKEN ([rows][d], y_dt).
 *   alpha, beta : finite; eps: finite, at least 1e-30.
 */
enum { TTT_GATE_NONE = 0, TTT_GATE_CHANNEL = 1, TTT_GATE_TOKEN = 2 };
int ttt_norm_pre(const void *h, ttt_dtype h_dt, const void *w, ttt_dtype w_dt, float eps, int64_t rows, int d, void *x,
                 ttt_dtype x_dt, void *hip_stream);
int ttt_norm_post(const void *h, ttt_dtype h_dt, const void *y, ttt_dtype y_dt, const void *w, const void *gate,
                  int gate_kind, const void *w_next, ttt_dtype w_dt, float alpha, float beta, float eps, int64_t rows,
                  int d, void *o, void *x, ttt_dtype x_dt, void *hip_stream);

/*
 * Their gradients.
 *
 *   ttt_norm_pre_grad  : from dx (the gradient of x) and dh_in (the gradient
 *                        of h from elsewhere, e.g. the residual path; NULL:
 *                        none) the gradient dh of h, dh_in included, and dw
 *                        ([d] fp32; NULL: not wanted).
 *   ttt_norm_post_grad : from dx (NULL: no norm followed, or no gradient came
 *                        through it) and dh_in (the gradient of o from
 *                        elsewhere; NULL: none; one of the two is needed), with
 *                        o as ttt_norm_post wrote it (read only with dx) and y:
 *                        dh [rows][d] (gradient of h), dy [rows][d], dw and
 *                        dw_next ([d] fp32), and dgate: [d] fp32 for a gate
 *                        per channel, [rows][d] of y's type for one per
 *                        token. dw, dw_next and dgate per channel may be NULL;
 *                        dgate per token may not. dw_next is not written
 *                        without dx.
 *
 * Rows as large as above are taken where |beta * gate * w| is at most 32 (the
 * formulas hold products beta * gate * w * y * o).
 *
 * dh has h_dt and may be dh_in (in place); dy has y_dt and may be y. The sums
 * over the rows are fp32, in an order fixed by rows, d and the types: the same
 * call gives the same bits. With rows = 0 the parameters' gradients are written as zero.
 * ws is needed when a parameter's gradient is wanted.
 */
int ttt_norm_ws_bytes(int64_t rows, int d, size_t *bytes);
int ttt_norm_pre_grad(const void *dx, ttt_dtype x_dt, const void *h, ttt_dtype h_dt, const void *w, ttt_dtype w_dt,
                      const void *dh_in, float eps, int64_t rows, int d, void *dh, float *dw, void *ws, size_t ws_bytes,
                      void *hip_stream);
int ttt_norm_post_grad(const void *dh_in, const void *dx, ttt_dtype x_dt, const void *o, ttt_dtype h_dt, const void *y,
                       ttt_dtype y_dt, const void *w, const void *gate, int gate_kind, const void *w_next,
                       ttt_dtype w_dt, float alpha, float beta, float eps, int64_t rows, int d, void *dh, void *dy,
                       float *dw, void *dgate, float *dw_next, void *ws, size_t ws_bytes, void *hip_stream);

/*
 * Token embedding and its gradient:
 *
 *   ttt_embed      : x[t] = scale * E[ids[t]], rounded once
 *   ttt_embed_grad : dE[v] = scale * sum of dx[t] over the tokens t with
 *                    ids[t] = v, summed in fp32, scaled and rounded. With
 *                    accumulate = 0 all of dE is written (zero rows for ids
 *                    that do not occur); otherwise the sums are added to the
 *                    rows that occur and the others are left alone.
 *
 * An id outside [0, vocab) gives a zero row and takes no gradient (its row of
 * dx is not read), like the zero target rows of the layer.
 *
 *   E, dE : [vocab][d], fp32 or bf16; vocab 1 .. 2^30, d 8 .. 65536.
 *   ids   : [B][T] int32, rows ids_ld >= T elements apart (so the [B][T+1] ids
 *           of ttt_forward_chunked serve with ids_ld = T + 1). B, T >= 0,
 *           B * T at most 2^27.
 *   x, dx : [B][T][d], fp32 or bf16, each independent of the table's type.
 *   scale : finite.
 *
 * The gradient sorts the tokens by id and sums each row's in the order of
 * their positions, a long row's in pieces of 32 that join in fp64 by eights:
 * the same call gives the same bits. ws: see ttt_embed_grad_ws_bytes (about 16 bytes per token, 8 per table
 * row and d / 4 bytes per token for the pieces).
 */
int ttt_embed(const void *E, ttt_dtype E_dt, int vocab, int d, const int32_t *ids, int64_t ids_ld, int B, int T,
              float scale, void *x, ttt_dtype x_dt, void *hip_stream);
int ttt_embed_grad_ws_bytes(int B, int T, int vocab, int d, size_t *bytes);
int ttt_embed_grad(const void *dx, ttt_dtype dx_dt, const int32_t *ids, int64_t ids_ld, int B, int T, float scale,
                   int vocab, int d, void *dE, ttt_dtype dE_dt, int accumulate, void *ws, size_t ws_bytes,
                   void *hip_stream);

/*
 * The global gradient norm over many tensors, and clipping by it:
 *
 *   ttt_grad_norm  : *norm = N = (sum over all tensors of g^2)^1/2
 *   ttt_clip_grads : the same, and out[i] = g[i] * min(1, tau / N)
 *
 * (The layer's own updates are clipped by ttt_set_clip.) Squares are summed in
 * fp64, in an order fixed by the sizes and types of the list and by which of
 * its neighbours adjoin in memory too (those are taken as one): the same call
 * gives the same bits, and both entry points the same norm, wherever outputs
 * lie. A norm that is not finite (a gradient holds an infinity or NaN) clips
 * nothing: the gradients come out as they are, and *norm says so. The host
 * learns of nothing and waits for nothing.
 *
 *   grads : host array of n device pointers; numel, dt: host arrays of their
 *           element counts (together at most 2^40) and types (ttt_dtype). The
 *           arrays may be freed on return. n 0 .. 2^20; n = 0 gives norm 0.
 *   out   : host array of n device pointers, each of its gradient's type and
 *           size, and each either the gradient itself (in place) or a copy
 *           that overlaps nothing; NULL: all in place. In place nothing is
 *           written unless the norm passes tau. A tensor may then not be
 *           listed twice (TTT_E_ARG); for the norm alone it may, and counts
 *           twice.
 *   tau   : greater than 0; +inf clips nothing.
 *   norm  : device, one float (inf where N is past fp32).
 *   ws    : device, ttt_grad_ws_bytes(n) bytes.
 */
int ttt_grad_ws_bytes(int n, size_t *bytes);
int ttt_grad_norm(const void *const *grads, const int64_t *numel, const int32_t *dt, int n, float *norm, void *ws,
                  size_t ws_bytes, void *hip_stream);
int ttt_clip_grads(const void *const *grads, const int64_t *numel, const int32_t *dt, int n, float tau,
                   void *const *out, float *norm, void *ws, size_t ws_bytes, void *hip_stream);

/*
 * The plain layers of a stack, whose MLPs do not learn at test time: a gated
 * feed-forward block is ttt_gated followed by ttt_linear with the residual
 * stream (paperlayer sec. 4: the fast weights stand in every 6th MLP). Rows
 * are tokens; x [rows][in], rows 0 .. 2^31-1, widths 1 .. 2^20.
 *
 *   a(p): TTT_ACT_NONE p; TTT_ACT_SILU p / (1 + e^-p); TTT_ACT_GELU the tanh
 *         form, p / (1 + e^-2w) with w = sqrt(2 / pi) (p + 0.044715 p^3);
 *         TTT_ACT_RELU max(p, 0).
 *
 *   ttt_linear : p = x W^T + bias,  y = residual + scale * a(p)
 *   ttt_gated  : g = x W_gate^T + b_gate,  u = x W_up^T + b_up,  z = a(g) * u
 *                (TTT_ACT_NONE is not taken)
 *
 *   W       : [out][in]; W_gate, W_up: [f][in].
 *   bias    : [out]; b_gate, b_up: [f], both or neither. NULL: none.
 *   residual: [rows][out] of y's type, or NULL. y may be the residual (in
 *             place).
 *   pre     : [rows][out], receives p; g, u: [rows][f], both or neither. NULL:
 *             not kept. The gradients need them (pre only with an activation).
 *   types   : dt is the type of x, the weights, the biases and what is kept
 *             (and of z); y and residual are fp32, or bf16 where dt is.
 *
 * bf16 products run on bf16 MFMA, fp32 ones on fp32 MFMA; sums are fp32, and
 * each result is rounded once, from fp32 values of what it depends on (y and z
 * from p, g and u as they were before they are rounded to be kept).
 */
enum { TTT_ACT_NONE = 0, TTT_ACT_SILU = 1, TTT_ACT_GELU = 2, TTT_ACT_RELU = 3 };
int ttt_linear_ws_bytes(int64_t rows, int in, int out, ttt_dtype dt, size_t *bytes);
int ttt_linear(const void *x, const void *W, ttt_dtype dt, const void *bias, int act, float scale,
               const void *residual, int64_t rows, int in, int out, void *pre, void *y, ttt_dtype y_dt, void *ws,
               size_t ws_bytes, void *hip_stream);
int ttt_gated_ws_bytes(int64_t rows, int in, int f, ttt_dtype dt, size_t *bytes);
int ttt_gated(const void *x, const void *W_gate, const void *W_up, ttt_dtype dt, const void *b_gate, const void *b_up,
              int act, int64_t rows, int in, int f, void *g, void *u, void *z, void *ws, size_t ws_bytes,
              void *hip_stream);

/*
 * Their gradients.
 *
 *   ttt_linear_grad : q = scale * dy * a'(pre);  dx = q W,  dW = q^T x,
 *                     dbias = the sum of q over the rows. (The residual's
 *                     gradient is dy itself.)
 *   ttt_gated_grad  : dg = dz * u * a'(g),  du = dz * a(g);
 *                     dx = dg W_gate + du W_up,  dW_gate = dg^T x,
 *                     dW_up = du^T x, db_gate, db_up the sums of dg, du
 *
 * dx, dW have dt; dbias, db_gate, db_up are fp32 ([out], [f]). Each may be
 * NULL (not wanted; dW_gate and dW_up, db_gate and db_up come in pairs). pre
 * is needed with an activation. With accumulate != 0 the weights' and biases'
 * gradients are added to what is there (gradients of several batches), dx is
 * always written. rows = 0 writes them as zero, or leaves them.
 *
 * The products of bf16 calls take q, dg and du as bf16, as their matrix
 * instructions do: one more rounding, half a step of each term, also of an fp32
 * dy. Beside the rounding of the results it makes the error of dx and dW 1.41
 * times what products of exact q would leave (in the mean square 0.0023 and
 * 0.0017 of the result); a caller who needs those takes the fp32 form, with x
 * and W in fp32. Where q is dy, in bf16 and without an activation, there is no
 * such rounding. The biases' gradients sum the unrounded ones. Every sum's order is
 * fixed by the sizes and types and by whether the operands start on 16 bytes
 * (the kernels for those that do are the faster ones): the same call gives the
 * same bits.
 *
 * ws holds q (or dg and du) where they are made, and fp32 sums of the biases'
 * gradients and of products whose k is split; operands of odd widths are copied
 * to it too where that pays. Its size: the _ws_bytes queries.
 */
int ttt_linear_grad_ws_bytes(int64_t rows, int in, int out, ttt_dtype dt, ttt_dtype y_dt, int act, size_t *bytes);
int ttt_linear_grad(const void *dy, ttt_dtype y_dt, const void *x, const void *W, ttt_dtype dt, const void *pre,
                    int act, float scale, int64_t rows, int in, int out, void *dx, void *dW, float *dbias,
                    int accumulate, void *ws, size_t ws_bytes, void *hip_stream);
int ttt_gated_grad_ws_bytes(int64_t rows, int in, int f, ttt_dtype dt, size_t *bytes);
int ttt_gated_grad(const void *dz, const void *x, const void *W_gate, const void *W_up, ttt_dtype dt, const void *g,
                   const void *u, int act, int64_t rows, int in, int f, void *dx, void *dW_gate, void *dW_up,
                   float *db_gate, float *db_up, int accumulate, void *ws, size_t ws_bytes, void *hip_stream);

/*
 * ttt_dense_plan — host-only query of how one product of the calls above runs
 * (no device work; usable without a GPU), for arrays that start on 16 bytes:
 *   q_made : for the two products of ttt_linear_grad: q is made, i.e. there is
 *            an activation or dy is not of type dt (0: dy itself serves).
 *   *kernel: TTT_KERNEL_FEW for up to 16 rows forward, TTT_KERNEL_DIRECT with
 *            tiles from memory straight to LDS, TTT_KERNEL_GENERAL through
 *            registers;  *tile: the tiles' side (0 with TTT_KERNEL_FEW);
 *   *splits: parts of k that are summed apart and joined by a second launch;
 *   *copies: matrices copied to rows of whole 16-byte pieces first.
 * Any output pointer may be NULL. Which sizes run how may change from one
 * version of the library to the next.
 */
enum {
  TTT_PRODUCT_LINEAR = 0,     /* ttt_linear: x W^T */
  TTT_PRODUCT_GATED = 1,      /* ttt_gated: x W_gate^T and x W_up^T */
  TTT_PRODUCT_LINEAR_DX = 2,  /* ttt_linear_grad: q W */
  TTT_PRODUCT_LINEAR_DW = 3,  /* q^T x */
  TTT_PRODUCT_GATED_DX = 4,   /* ttt_gated_grad: dg W_gate + du W_up */
  TTT_PRODUCT_GATED_DW = 5    /* dg^T x and du^T x */
};
enum { TTT_KERNEL_FEW = 0, TTT_KERNEL_DIRECT = 1, TTT_KERNEL_GENERAL = 2 };
int ttt_dense_plan(int product, int64_t rows, int in, int out, ttt_dtype dt, int q_made, int *kernel, int *tile,
                   int *splits, int *copies);

/*
 * ttt_adamw — one AdamW step over many tensors:
 *
 *   g' = g * min(1, tau / N)                    (norm not NULL: N = *norm)
 *   m' = beta1 m + (1 - beta1) g',  v' = beta2 v + (1 - beta2) g'^2
 *   w' = w (1 - lr weight_decay) - lr (m' / (1 - beta1^step)) / (sqrt(v' / (1 - beta2^step)) + eps)
 *
 *   w, g    : host arrays of n device pointers, w_dt, g_dt their types (fp32
 *             or bf16, each its own), numel their element counts (together at
 *             most 2^40). The arrays may be freed on return. n 0 .. 2^20.
 *   m, v    : the moments, in place: fp32 (state_bits 32) or codes of 8 bits,
 *             a byte each (state_bits 8). All bytes zero: moments of zero.
 *   tops    : state_bits 8: per tensor [2][ceil(numel / 256)] int16 (m's row,
 *             then v's), zero at the start. NULL with state_bits 32.
 *   copies  : NULL, or n pointers to bf16 arrays (or NULL) that receive w'
 *             rounded, for an fp32 w whose next forward pass runs in bf16.
 *   step    : 1, 2, ...; read from step_dev (device, one int64) where that is
 *             not NULL, as lr is from lr_dev (device, one float), so that a
 *             captured call can be replayed with others.
 *   norm    : device, one float, as ttt_grad_norm or ttt_clip_grads gives it,
 *             or NULL. One that is not finite clips nothing. tau > 0.
 *   beta1, beta2 : in [0, 1); eps, weight_decay: finite, not negative; lr:
 *             finite.
 *
 * 8-bit moments. T, a block's top (256 elements from the tensor's start), is
 * the least multiple of 2^20, in units of 2^20, that no |x| of the block passes
 * as an fp32 bit pattern. m's code is a sign (bit 7) and c in 0 .. 127, v's is
 * c in 0 .. 255; c > 0 stands for the fp32 number of pattern (T - most + c)
 * << 20, most = 127 or 255 (0 where that is not positive), c = 0 for 0: three
 * mantissa bits over the 16 (32) octaves under the block's largest. m' and v'
 * are computed in fp64, rounded to fp32 and then to one of the two neighbouring
 * codes at random, so that the expectation is kept: of |x|'s pattern P, (P +
 * 16 r) >> 20 with 16 random bits r; below the smallest value s of the block m'
 * becomes s where |m'| >= (r + 1/2) 2^-16 s and 0 otherwise, and a v' that is
 * not 0 becomes s. r is the low half for m, the high half for v, of 32 bits
 * made of seed, step, the tensor's number in the list and the element's number
 * in the tensor (modulo 2^32): the same call gives the same codes. w' is
 * computed from the moments before they become codes.
 *
 * Every array but g may be written; none may overlap another (TTT_E_ARG).
 *
 * ttt_adamw_values — the fp32 values of codes: moment 1 (codes m, first row of
 * tops) or 2.
 */
int ttt_adamw(void *const *w, const int32_t *w_dt, const void *const *g, const int32_t *g_dt, void *const *m,
              void *const *v, int state_bits, int16_t *const *tops, void *const *copies, const int64_t *numel, int n,
              int64_t step, const int64_t *step_dev, double lr, const float *lr_dev, double beta1, double beta2,
              double eps, double weight_decay, const float *norm, double tau, uint32_t seed, void *hip_stream);
int ttt_adamw_values(const void *const *codes, const int16_t *const *tops, int moment, float *const *out,
                     const int64_t *numel, int n, void *hip_stream);

#ifdef __cplusplus
}
#endif
#endif /* TTT_H */

"""The operators around the layer, run together with it as a stack runs them: token embedding, the norm before the first
layer, layers with the norm after each (and the next one's before it), and back: the norms' gradients, the embedding's,
and one clipping over all of them."""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as ttt
import oracle
from synth import make_inputs
from tests.block_util import U32, assert_close, half_step, rms64
from tests.gpu_util import dev, max_rel, rel_fro, torch_dtype

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(dtype, layers, seed, eta):
    d, f = (256, 512) if dtype == "bf16" else (64, 256)
    ws = [make_inputs(d=d, f=f, B=2, T=700, C=128, eta=eta, dtype=dtype, vocab=300, e_std=1.0, seed=seed + k)
          for k in range(layers)]
    g = torch.Generator().manual_seed(seed)
    gains = [{k: torch.randn(d, generator=g) * 0.2 + (0.5 if k == "gate" else 1.0) for k in ("pre", "post", "gate")}
             for _ in range(layers)]
    return ws, gains


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_stack_forward_with_learning_layers(dtype):
    """Every stage against 64 bits on the inputs it was given: the layers against the oracle within its bars, the
    operators within their own bounds (their rounding and 512 fp32 roundings at most)."""
    ws, gains = make(dtype, 2, 40, 2e-3)
    dt = torch_dtype(ws[0])
    w0 = ws[0]
    ids = torch.from_numpy(w0.ids).cuda()
    E = dev(w0.E_tgt, dt)
    h = ttt.ttt_embed(E, ids[:, :-1], scale=float(np.sqrt(w0.d)), dtype=torch.float32)
    want = E.double()[ids[:, :-1].long()] * float(np.float32(np.sqrt(w0.d)))
    assert_close(h, want.cpu(), 4 * U32 * want.abs().cpu(), "embedding")
    x = ttt.ttt_norm_pre(h, gains[0]["pre"].cuda(), eps=EPS, dtype=dt)
    want = gains[0]["pre"].double().cuda() * h.double() * rms64(h.double(), EPS)
    assert_close(x, want.cpu(), ((512 * U32 + 1.01 * half_step(dt)) * want.abs()).cpu(), "first norm")
    for k, w in enumerate(ws):
        layer = ttt.ttt_init(dev(w.W_up, dt), dev(w.W_gate, dt), dev(w.W_down0, dt), w.C, w.eta, max_batch=w.B)
        y, Wf = ttt.ttt_forward_chunked(layer, x, ids, E, want_W_final=True)
        y_ref, W_ref = oracle.ttt_forward(x.double().cpu().numpy(), w0.ids, w0.E_tgt, w.W_up, w.W_gate, w.W_down0, w.C,
                                          w.eta)
        metric, tol = (rel_fro, 3e-2) if dtype == "bf16" else (max_rel, 1e-4)
        assert metric(y.double().cpu().numpy(), y_ref) <= tol
        assert metric(Wf.double().cpu().numpy(), W_ref) <= tol
        last = k + 1 == len(ws)
        nxt = None if last else gains[k + 1]["pre"].cuda()
        before = h.clone()
        h, x = ttt.ttt_norm_post(h, y, gains[k]["post"].cuda(), gate=gains[k]["gate"].cuda(), beta=0.5, eps=EPS,
                                 w_next=nxt, o=h, dtype=dt)
        branch = 0.5 * (gains[k]["gate"] * gains[k]["post"]).double().cuda() * y.double() * rms64(y.double(), EPS)
        o = before.double() + branch
        bound = 512 * U32 * (before.double().abs() + branch.abs())
        assert_close(h, o.cpu(), (bound + U32 * o.abs()).cpu(), "stream")
        if last:
            assert x is None
        else:
            r = rms64(o, EPS)
            want = nxt.double() * o * r
            norm = o.norm(dim=-1, keepdim=True)
            b = nxt.double().abs() * r * (bound + o.abs() * (bound.norm(dim=-1, keepdim=True) / norm + 512 * U32))
            assert_close(x, want.cpu(), (b + half_step(dt) * (want.abs() + b)).cpu(), "next norm")
        ttt.ttt_destroy(layer)


def test_training_step_against_autograd():
    """Gradients of a two-layer stack whose layers do not learn (eta = 0: a static gated MLP, differentiated by torch in
    64 bits on the layer's own inputs), clipped together, against autograd of the whole model in 64 bits.

    Bound: the layer's bar is 1e-4 of its largest value and the operators lie far below it; two layers and three norms
    each way make ten stages, and a product passes on the relative errors of both its factors: 2 * 10 * 1e-4 = 2e-3 of
    the largest value. This is a test of how the parts meet; each part's own bounds are tested apart."""
    ws, gains = make("f32", 2, 60, 0.0)
    w0 = ws[0]
    d, scale, beta = w0.d, 8.0, 0.5
    ids = torch.from_numpy(w0.ids).cuda()
    E = dev(w0.E_tgt, torch.float32)
    gen = torch.Generator().manual_seed(1)
    target = torch.randn((w0.B, w0.T, d), generator=gen).cuda() / (w0.B * w0.T)
    G = [{k: v.cuda() for k, v in g.items()} for g in gains]

    # forward, keeping what the gradients need
    h = ttt.ttt_embed(E, ids[:, :-1], scale=scale)
    emb = h
    x = ttt.ttt_norm_pre(h, G[0]["pre"], eps=EPS)
    kept = []
    for k, w in enumerate(ws):
        layer = ttt.ttt_init(dev(w.W_up, torch.float32), dev(w.W_gate, torch.float32), dev(w.W_down0, torch.float32),
                             w.C, w.eta, max_batch=w.B)
        y, _ = ttt.ttt_forward_chunked(layer, x, ids, E)
        nxt = G[k + 1]["pre"] if k == 0 else None
        o, x_next = ttt.ttt_norm_post(h, y, G[k]["post"], gate=G[k]["gate"], beta=beta, eps=EPS, w_next=nxt)
        kept.append((x, y, o))
        h, x = o, x_next
        ttt.ttt_destroy(layer)

    def mlp(w, x64):
        up, gate, down = (torch.from_numpy(np.asarray(t)).double().cuda() for t in (w.W_up, w.W_gate, w.W_down0))
        return (torch.nn.functional.silu(x64 @ gate.t()) * (x64 @ up.t())) @ down.t()

    # backward of the loss <h, target>
    names, grads = [], []
    dh, dx = target, None
    for k in (1, 0):
        x_in, y, o = kept[k]
        nxt = G[1]["pre"] if k == 0 else None
        g = ttt.ttt_norm_post_grad(dh, dx, o, y, G[k]["post"], gate=G[k]["gate"], beta=beta, eps=EPS, w_next=nxt)
        names += [("post", k), ("gate", k)]
        grads += [g.dw, g.dgate]
        if k == 0:
            names.append(("pre", 1))
            grads.append(g.dw_next)
        x64 = x_in.double().requires_grad_()
        dx = torch.autograd.grad(mlp(ws[k], x64), x64, g.dy.double())[0].float()
        dh = g.dh
    dh, dpre = ttt.ttt_norm_pre_grad(dx, emb, G[0]["pre"], eps=EPS, dh_in=dh)
    dE = ttt.ttt_embed_grad(dh, ids[:, :-1], w0.vocab, scale=scale)
    names += [("pre", 0), ("E", 0)]
    grads += [dpre, dE]

    # the same model in 64 bits
    E64 = E.double().requires_grad_()
    P = [{k: v.double().requires_grad_() for k, v in g.items()} for g in G]
    s = E64[ids[:, :-1].long()] * scale
    z = P[0]["pre"] * s * rms64(s, EPS)
    for k, w in enumerate(ws):
        y64 = mlp(w, z)
        s = s + beta * P[k]["gate"] * P[k]["post"] * y64 * rms64(y64, EPS)
        if k == 0:
            z = P[1]["pre"] * s * rms64(s, EPS)
    leaves = [E64 if n == "E" else P[k][n] for n, k in names]
    want = torch.autograd.grad((s * target.double()).sum(), leaves)
    for (n, k), a, b in zip(names, grads, want):
        assert max_rel(a.double().cpu().numpy(), b.cpu().numpy()) <= 2e-3, (n, k)

    # one clipping over all of them
    n64 = float(torch.sqrt(sum(b.square().sum() for b in want)))
    got = [g.clone() for g in grads]
    norm = ttt.ttt_clip_grads(got, 0.25 * n64)
    assert abs(float(norm) - n64) <= 2e-3 * n64
    for a, b in zip(got, grads):
        ref = b.double() * (float(np.float32(0.25 * n64)) / float(norm))
        assert_close(a, ref.cpu(), 4 * U32 * ref.abs().cpu(), "clipped")
    assert abs(float(ttt.ttt_grad_norm(got)) - 0.25 * n64) <= 1e-5 * n64


def test_decoding_step_in_a_graph():
    """One token per sequence through embedding, norms and a layer, captured once (the layer by its call that allocates
    nothing) and replayed with new tokens between eager work: each replay equals the eager run bit for bit."""
    ws, gains = make("bf16", 1, 80, 0.0)
    w = ws[0]
    E = dev(w.E_tgt, torch.bfloat16)
    layer = ttt.ttt_init(dev(w.W_up, torch.bfloat16), dev(w.W_gate, torch.bfloat16), dev(w.W_down0, torch.bfloat16),
                         w.C, 0.0, max_batch=w.B)
    G = {k: v.cuda() for k, v in gains[0].items()}
    ids = torch.zeros((w.B, 2), dtype=torch.int32, device="cuda")
    y = torch.empty((w.B, 1, w.d), dtype=torch.bfloat16, device="cuda")

    def step():
        h = ttt.ttt_embed(E, ids[:, :1], scale=4.0, dtype=torch.float32)
        x = ttt.ttt_norm_pre(h, G["pre"], dtype=torch.bfloat16)
        ttt.ttt_forward_chunked_noalloc(layer, x, ids, E, y)
        return ttt.ttt_norm_post(h, y, G["post"], gate=G["gate"], w_next=G["pre"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        ids.copy_(torch.from_numpy(w.ids[:, k:k + 2].copy()).cuda())
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out)), k
    ttt.ttt_destroy(layer)

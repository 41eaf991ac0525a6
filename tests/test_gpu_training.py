"""The plain layers, the norms, the embedding, the clipping and the AdamW step run together as a stack trains and serves."""
import math

import pytest
import torch

import chunk_wise_weight_amd as ttt
from synth import make_inputs
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu
EPS = 1e-6
HYPER = dict(betas=(0.9, 0.95), eps=1e-8, weight_decay=0.05)
F32, BF16 = torch.float32, torch.bfloat16


class Stack:
    """ids -> embedding -> layers of (norm, gated projections, down projection into the stream) -> a last norm."""

    def __init__(self, layers, vocab, d, f, dt, seed):
        g = torch.Generator().manual_seed(seed)

        def make(*shape, std=1.0, mean=0.0):
            return (torch.randn(shape, generator=g) * std + mean).to(dt).cuda()

        self.scale = math.sqrt(d)
        self.params = [make(vocab, d, std=0.1)]
        for _ in range(layers):
            self.params += [make(d, std=0.1, mean=1.0), make(f, d, std=d ** -0.5), make(f, d, std=d ** -0.5),
                            make(f, std=0.1), make(f, std=0.1), make(d, f, std=f ** -0.5), make(d, std=0.1)]
        self.params.append(make(d, std=0.1, mean=1.0))
        self.layers, self.dt = layers, dt

    def forward(self, ids):
        P, dt = self.params, self.dt
        h = ttt.ttt_embed(P[0], ids, scale=self.scale, dtype=F32)
        kept = []
        for k in range(self.layers):
            w, wg, wu, bg, bu, wd, bd = P[1 + 7 * k:8 + 7 * k]
            x = ttt.ttt_norm_pre(h, w, eps=EPS, dtype=dt)
            z, g, u = ttt.ttt_gated(x, wg, wu, bg, bu, keep=True)
            out = ttt.ttt_linear(z, wd, bd, residual=h)
            kept.append((h, x, z, g, u))
            h = out
        return h, ttt.ttt_norm_pre(h, P[-1], eps=EPS), kept

    def backward(self, ids, dx, h, kept):
        P = self.params
        dh, dw = ttt.ttt_norm_pre_grad(dx, h, P[-1], eps=EPS)
        grads = [None] * len(P)
        grads[-1] = dw
        for k in reversed(range(self.layers)):
            w, wg, wu, _, _, wd, _ = P[1 + 7 * k:8 + 7 * k]
            h, x, z, g, u = kept[k]
            lin = ttt.ttt_linear_grad(dh, z, wd, bias=True)
            gat = ttt.ttt_gated_grad(lin.dx, x, wg, wu, g, u, bias=True)
            dh, dw = ttt.ttt_norm_pre_grad(gat.dx, h, w, eps=EPS, dh_in=dh)
            grads[1 + 7 * k:8 + 7 * k] = [dw, gat.dw_gate, gat.dw_up, gat.db_gate, gat.db_up, lin.dw, lin.dbias]
        grads[0] = ttt.ttt_embed_grad(dh, ids, P[0].shape[0], scale=self.scale, dtype=F32)
        return grads


def forward64(params, ids, layers, scale):
    def norm(h, w):
        return w * h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)

    h = params[0][ids.long()] * scale
    for k in range(layers):
        w, wg, wu, bg, bu, wd, bd = params[1 + 7 * k:8 + 7 * k]
        x = norm(h, w)
        g = x @ wg.T + bg
        h = h + (g * torch.sigmoid(g) * (x @ wu.T + bu)) @ wd.T + bd
    return norm(h, params[-1])


@pytest.mark.parametrize("dt,T,d,f", [(F32, 37, 72, 100), (F32, 150, 64, 200), (BF16, 300, 128, 264)])
def test_three_steps_against_64_bits(dt, T, d, f):
    """Gradients and the weights after each step against autograd and the formula in 64 bits, the 64-bit side starting each
    step from the weights and moments the other side has. fp32: two layers of products and three norms each way, every
    stage within 10^-6 of its largest value, so 10^-4 of a gradient's norm has room. bf16: a stage's roundings are 2^-9
    of each value, independent, with ten stages in a row: 4 % of a gradient's norm."""
    layers, vocab = 2, 50
    net = Stack(layers, vocab, d, f, dt, 3)
    gen = torch.Generator().manual_seed(1)
    ids = torch.randint(0, vocab, (2, T), generator=gen).int().cuda()
    target = torch.randn((2, T, d), generator=gen).cuda()
    m, v = ([torch.zeros_like(p, dtype=F32) for p in net.params] for _ in range(2))
    for step in range(1, 4):
        before = [p.double().clone() for p in net.params]
        om, ov = [t.double() for t in m], [t.double() for t in v]
        h, out, kept = net.forward(ids)
        grads = net.backward(ids, (out - target) / out.numel(), h, kept)
        leaves = [p.requires_grad_() for p in before]
        y = forward64(leaves, ids, layers, net.scale)
        loss = 0.5 * ((y - target.double()) ** 2).sum() / y.numel()
        want = torch.autograd.grad(loss, leaves)
        tol = 1e-4 if dt == F32 else 0.04
        for i, (a, b) in enumerate(zip(grads, want)):
            assert float((a.double() - b).norm()) <= tol * float(b.norm()), (step, i)
        norm = ttt.ttt_grad_norm(grads)
        tau = 0.5 * float(norm)
        copies = [torch.empty_like(p, dtype=BF16) for p in net.params]
        ttt.ttt_adamw(net.params, grads, m, v, step, 1e-2, copies=copies, norm=norm, tau=tau, **HYPER)
        b1, b2 = HYPER["betas"]
        for i, p in enumerate(net.params):
            g = grads[i].double() * (tau / float(norm.double()))
            m1, v1 = b1 * om[i] + (1 - b1) * g, b2 * ov[i] + (1 - b2) * g * g
            w1 = before[i].detach() * (1 - 1e-2 * HYPER["weight_decay"]) - 1e-2 * (m1 / (1 - b1 ** step)) / (
                torch.sqrt(v1 / (1 - b2 ** step)) + HYPER["eps"])
            # a rounding to the weight's type, and the step (at most 10 lr here) to 10^-5
            assert bool(((p.double() - w1).abs() <= torch.finfo(dt).eps / 2 * 1.01 * w1.abs() + 1e-6).all()), (step, i)
            assert bool(((copies[i].double() - w1).abs() <= 2.0 ** -8 * 1.02 * w1.abs() + 1e-6).all())


def test_training_step_in_a_graph():
    """A whole step, forward to the weights, captured once and replayed with the step and the rate on the device, against
    the same calls made one by one."""
    layers, vocab, d, f, T = 2, 40, 64, 136, 90
    gen = torch.Generator().manual_seed(2)
    ids = torch.randint(0, vocab, (3, T), generator=gen).int().cuda()
    target = torch.randn((3, T, d), generator=gen).cuda()

    def make():
        net = Stack(layers, vocab, d, f, F32, 5)
        c = [torch.zeros_like(p, dtype=torch.uint8) for p in net.params]
        e = [torch.zeros_like(p, dtype=torch.uint8) for p in net.params]
        tops = [torch.zeros((2, -(-p.numel() // 256)), dtype=torch.int16, device="cuda") for p in net.params]
        return net, c, e, tops

    def step(s, t, lr):
        net, c, e, tops = s
        h, out, kept = net.forward(ids)
        grads = net.backward(ids, (out - target) / out.numel(), h, kept)
        norm = ttt.ttt_grad_norm(grads)
        ttt.ttt_adamw(net.params, grads, c, e, t, lr, tops=tops, seed=7, norm=norm, tau=0.05, **HYPER)
        return norm

    a, b = make(), make()
    t, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.full((1,), 1e-2, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(make(), t, lr)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm = step(a, t, lr)
    for k in range(1, 5):
        t.fill_(k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step(b, k, float(lr))
        assert torch.equal(norm, want)
        for p, q in zip(a[0].params + a[1] + a[2] + a[3], b[0].params + b[1] + b[2] + b[3]):
            assert torch.equal(p, q), k


def test_decoding_with_a_learning_layer():
    """Tokens one at a time through a plain layer, a layer that learns and the norms around them, the stream updated in
    place: each token's plain layers give what the whole sequence at once gives, to their roundings."""
    w = make_inputs(d=256, f=512, B=2, T=24, C=8, eta=0.0, dtype="bf16", vocab=64, e_std=1.0, seed=5)
    ids = torch.from_numpy(w.ids).cuda()
    E = dev(w.E_tgt, BF16)
    g = torch.Generator().manual_seed(3)
    wg, wu, wd = ((torch.randn(s, generator=g) * k).to(BF16).cuda() for s, k in
                  (((520, 256), 1 / 16), ((520, 256), 1 / 16), ((256, 520), 520 ** -0.5)))

    def run(ids, layer):
        h = ttt.ttt_embed(E, ids[:, :-1], dtype=F32)
        z = ttt.ttt_gated(ttt.ttt_norm_pre(h, eps=EPS, dtype=BF16), wg, wu)
        h = ttt.ttt_linear(z, wd, residual=h, y=h)
        x = ttt.ttt_norm_pre(h, eps=EPS, dtype=BF16)
        y, _ = ttt.ttt_forward_chunked(layer, x, ids, E)
        return ttt.ttt_norm_post(h, y, o=h)[0]

    def layer():
        return ttt.ttt_init(dev(w.W_up, BF16), dev(w.W_gate, BF16), dev(w.W_down0, BF16), w.C, 0.0, max_batch=2)

    whole = run(ids, layer())
    one = layer()
    for t in range(w.T):
        got = run(ids[:, t:t + 2].contiguous(), one)
        # the stream is fp32; what differs are bf16 roundings of the layers' inputs and results: 2^-8 of values near 1
        assert float((got[:, 0] - whole[:, t]).norm()) <= 2e-2 * float(whole[:, t].norm()), t

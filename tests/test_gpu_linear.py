"""The plain layers' operators against their formulas in 64 bits: the matrix product with bias, activation and residual,
the gated projections, and the gradients of both.

Bounds, element by element. A sum of n products of which the magnitudes add up to S is off by at most (n + 2) roundings
of fp32, each U = 2^-24 of at most S; twice that leaves room for a matrix instruction that rounds inside. An activation
has |a'| <= 1.13, passing on its argument's error times 1.2, and its own error is below 16 U |p|: e^-e is off by (|e| + 4)
2^-23 relative with e = p or 2w, which reaches a = p h through h (1 - h) |e| <= 0.28 and h (1 - h) <= 1/4, and h itself
by a few U. A derivative (at most 1.13, h + p h (1 - h) slope) is off by 64 U: |p| h (1 - h) slope |e| <= 3, over the
same 2^-23 (|e| + 4)/|e|, and its own few products. A result then is rounded once to its type, and q, dg and du once
more to the products' type."""
import math

import pytest
import torch

import chunk_wise_weight_amd as ttt
from chunk_wise_weight_amd import binding
from tests.block_util import U32, assert_close, half_step

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
C0, C1 = math.sqrt(2 / math.pi), 0.044715


def act64(p, act):
    if act is None:
        return p
    if act == "relu":
        return p.clamp(min=0)
    e = p if act == "silu" else 2 * C0 * (p + C1 * p ** 3)
    return p * torch.sigmoid(e)


def d_act64(p, act):
    p = p.clone().requires_grad_()
    return torch.autograd.grad(act64(p, act).sum(), p)[0]


class Held:
    """A device array between two stretches of NaN, `off` elements into its buffer; check() looks that they are still
    there. What a kernel reads outside shows as NaN."""

    def __init__(self, t, off):
        n = t.numel()
        self.buf = torch.full((n + off + 64,), float("nan"), dtype=t.dtype, device="cuda")
        self.off, self.n = off, n
        self.t = self.buf[off:off + n].view(t.shape)
        self.t.copy_(t)

    def check(self):
        assert bool(self.buf[:self.off].isnan().all()) and bool(self.buf[self.off + self.n:].isnan().all())


def make(shape, dtype, g, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def empty(shape, dtype, off):
    return Held(torch.full(shape, 3.25, dtype=dtype), off)


# rows, in, out: one element, one row, odd widths, widths of 8 and 64, sides of the tiles, few rows and long sums
SIZES = [(1, 1, 1), (1, 9, 5), (2, 64, 7), (3, 7, 130), (129, 257, 131), (127, 64, 128), (1, 1024, 512), (5, 2560, 264),
         (16, 512, 96), (17, 328, 1000), (33, 520, 72), (64, 4096, 40), (65, 96, 320), (200, 96, 320), (257, 1000, 264),
         (513, 200, 520), (640, 1088, 776)]
OFFS = [0, 3]


def linear_case(M, K, N, dt, ydt, act, bias, res, scale, off):
    g = torch.Generator().manual_seed(M * 7 + K * 3 + N + off)
    x, w = make((M, K), dt, g), make((N, K), dt, g, K ** -0.5)
    b = make((N,), dt, g, 0.3) if bias else None
    r = make((M, N), ydt, g, 2.0) if res else None
    held = [Held(t, off) for t in (x, w)]
    hb, hr = (None if t is None else Held(t, off) for t in (b, r))
    y = empty((M, N), ydt, off)
    got, pre = ttt.ttt_linear(held[0].t, held[1].t, None if hb is None else hb.t, act=act,
                              residual=None if hr is None else hr.t, scale=scale, keep=True, y=y.t)
    assert got is y.t
    y.check()
    xd, wd = x.double(), w.double()
    p = xd @ wd.T
    S = xd.abs() @ wd.abs().T
    if bias:
        p, S = p + b.double(), S + b.double().abs()
    ep = 2 * (K + 3) * U32 * S
    assert_close(pre, p, ep + half_step(dt) * (p.abs() + ep), "pre")
    want = scale * act64(p, act)
    err = abs(scale) * (1.2 * ep + (16 * U32 * p.abs() if act else 0)) + 2 * U32 * want.abs()
    if res:
        want = want + r.double()
    err = err + U32 * want.abs()
    assert_close(y.t, want, err + half_step(ydt) * (want.abs() + err), "y")
    if ydt == F32 and act is None:
        # over many elements the roundings do not all point one way
        off_by = (y.t.double().cpu() - want).norm() / want.norm()
        assert off_by <= 4 * math.sqrt(K + 3) * U32, off_by


@pytest.mark.parametrize("off", OFFS)
@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("dt,ydt", [(F32, F32), (BF16, F32), (BF16, BF16)])
def test_linear(M, K, N, dt, ydt, off):
    linear_case(M, K, N, dt, ydt, None, False, False, 1.0, off)
    linear_case(M, K, N, dt, ydt, "gelu", True, True, 0.5, off)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "relu"])
@pytest.mark.parametrize("bias,res", [(False, True), (True, False)])
def test_linear_epilogues(act, bias, res):
    for M in (2, 100, 300):
        linear_case(M, 136, 200, BF16, BF16, act, bias, res, -2.0, 0)
        linear_case(M, 136, 200, F32, F32, act, bias, res, 1.0, 0)


def test_linear_in_place_residual():
    g = torch.Generator().manual_seed(1)
    for M in (1, 70, 700):
        x, w = make((M, 256), BF16, g).cuda(), make((320, 256), BF16, g, 1 / 16).cuda()
        h = make((M, 320), F32, g).cuda()
        want = ttt.ttt_linear(x, w, residual=h)
        got = ttt.ttt_linear(x, w, residual=h, y=h)
        assert got is h and torch.equal(got, want) and got.dtype == F32


def gated_case(M, K, f, dt, act, bias, off):
    g = torch.Generator().manual_seed(M * 5 + K + f + off)
    x, wg, wu = make((M, K), dt, g), make((f, K), dt, g, K ** -0.5), make((f, K), dt, g, K ** -0.5)
    bg, bu = (make((f,), dt, g, 0.3), make((f,), dt, g, 0.3)) if bias else (None, None)
    held = [Held(t, off).t for t in (x, wg, wu)]
    hb = [None if t is None else Held(t, off).t for t in (bg, bu)]
    z = empty((M, f), dt, off)
    got, kg, ku = ttt.ttt_gated(*held, *hb, act=act, keep=True, z=z.t)
    z.check()
    xd = x.double()
    G, U = xd @ wg.double().T, xd @ wu.double().T
    SG, SU = xd.abs() @ wg.double().abs().T, xd.abs() @ wu.double().abs().T
    if bias:
        G, U, SG, SU = G + bg.double(), U + bu.double(), SG + bg.double().abs(), SU + bu.double().abs()
    eg, eu = 2 * (K + 3) * U32 * SG, 2 * (K + 3) * U32 * SU
    assert_close(kg, G, eg + half_step(dt) * (G.abs() + eg), "g")
    assert_close(ku, U, eu + half_step(dt) * (U.abs() + eu), "u")
    a = act64(G, act)
    ea = 1.2 * eg + 16 * U32 * G.abs()
    want = a * U
    err = ea * U.abs() + (a.abs() + ea) * eu + 2 * U32 * want.abs()
    assert_close(z.t, want, err + half_step(dt) * (want.abs() + err), "z")
    alone = ttt.ttt_gated(*held, *hb, act=act)
    assert torch.equal(alone, z.t)


@pytest.mark.parametrize("off", OFFS)
@pytest.mark.parametrize("M,K,f", SIZES)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_gated(M, K, f, dt, off):
    gated_case(M, K, f, dt, "silu", False, off)
    gated_case(M, K, f, dt, "gelu", True, off)


def check_products(q, eq, x, w, dx, dw, dt, scale=1.0, extra=None):
    """dx = sum of q w and dw = q^T x over lists of (q, its error) and weights, elementwise bounds."""
    want = sum(a @ b.double() for a, b in zip(q, w)) * scale
    n = sum(a.shape[1] for a in q)
    err = sum((e + 2 * (n + 3) * U32 * (a.abs() + e)) @ b.double().abs() for a, e, b in zip(q, eq, w)) * abs(scale)
    err = err + 2 * U32 * want.abs()
    assert_close(dx, want, err + half_step(dt) * (want.abs() + err), "dx")
    M = x.shape[0]
    for i, (a, e, got) in enumerate(zip(q, eq, dw)):
        want = a.T @ x.double() * scale
        err = (e + 2 * (M + 3) * U32 * (a.abs() + e)).T @ x.double().abs() * abs(scale) + 2 * U32 * want.abs()
        if extra is not None:
            want = want + extra[i].double()
            err = err + U32 * want.abs()
        assert_close(got, want, err + half_step(dt) * (want.abs() + err), "dw")


def linear_grad_case(M, K, N, dt, ydt, act, scale, off, accumulate=False):
    g = torch.Generator().manual_seed(M * 3 + K * 5 + N + off)
    x, w = make((M, K), dt, g), make((N, K), dt, g, K ** -0.5)
    dy = make((M, N), ydt, g)
    pre = make((M, N), dt, g, 2.0) if act else None
    hx, hw, hy = Held(x, off), Held(w, off), Held(dy, off)
    hp = None if pre is None else Held(pre, off).t
    dx, dw, db = empty((M, K), dt, off), empty((N, K), dt, off), empty((N,), F32, off)
    got = ttt.ttt_linear_grad(hy.t, hx.t, hw.t, act=act, pre=hp, scale=scale, bias=True, dx=dx.t, dw=dw.t, dbias=db.t,
                              accumulate=accumulate)
    assert got.dx is dx.t and got.dw is dw.t and got.dbias is db.t
    for t in (dx, dw, db):
        t.check()
    q = dy.double() * (d_act64(pre.double(), act) if act else 1.0)
    eq = 64 * U32 * dy.double().abs() + 2 * U32 * q.abs() if act else torch.zeros_like(q)
    rounded = act or ydt != dt
    ep = eq + (half_step(dt) * (q.abs() + eq) if rounded else 0)
    old = [torch.full((N, K), 3.25)] if accumulate else None
    # with a pass of its own the scale is in q, else it multiplies the products: one rounding either way
    check_products([q], [ep + 2 * U32 * q.abs()], x, [w], dx.t, [dw.t], dt, scale, old)
    want = scale * q.sum(0)
    err = abs(scale) * (eq + 2 * U32 * q.abs() + 2 * (M + 3) * U32 * q.abs()).sum(0)
    if accumulate:
        want = want + 3.25
    assert_close(db.t, want, err + 2 * U32 * want.abs(), "dbias")


@pytest.mark.parametrize("off", OFFS)
@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("dt,ydt", [(F32, F32), (BF16, F32), (BF16, BF16)])
def test_linear_grad(M, K, N, dt, ydt, off):
    linear_grad_case(M, K, N, dt, ydt, None, 0.5, off)
    linear_grad_case(M, K, N, dt, ydt, "silu", 1.0, off, accumulate=True)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_linear_grad_activations(act):
    for dt in (F32, BF16):
        linear_grad_case(150, 72, 136, dt, dt, act, -2.0, 0)


def gated_grad_case(M, K, f, dt, act, off, accumulate=False):
    gen = torch.Generator().manual_seed(M + K * 5 + f + off)
    x, wg, wu = make((M, K), dt, gen), make((f, K), dt, gen, K ** -0.5), make((f, K), dt, gen, K ** -0.5)
    dz, g, u = make((M, f), dt, gen), make((M, f), dt, gen, 2.0), make((M, f), dt, gen)
    args = [Held(t, off).t for t in (dz, x, wg, wu, g, u)]
    outs = [empty(s, d, off) for s, d in (((M, K), dt), ((f, K), dt), ((f, K), dt), ((f,), F32), ((f,), F32))]
    ttt.ttt_gated_grad(*args, act=act, bias=True, dx=outs[0].t, dw_gate=outs[1].t, dw_up=outs[2].t, db_gate=outs[3].t,
                       db_up=outs[4].t, accumulate=accumulate)
    for t in outs:
        t.check()
    gd, ud, zd = g.double(), u.double(), dz.double()
    q = [zd * ud * d_act64(gd, act), zd * act64(gd, act)]
    e = [64 * U32 * (zd * ud).abs() + 3 * U32 * q[0].abs(), 16 * U32 * (zd * gd).abs() + 2 * U32 * q[1].abs()]
    er = [b + half_step(dt) * (a.abs() + b) for a, b in zip(q, e)]
    old = [torch.full((f, K), 3.25)] * 2 if accumulate else None
    check_products(q, er, x, [wg, wu], outs[0].t, [outs[1].t, outs[2].t], dt, extra=old)
    for a, b, t in zip(q, e, outs[3:]):
        want = a.sum(0) + (3.25 if accumulate else 0)
        err = (b + 2 * (M + 3) * U32 * (a.abs() + b)).sum(0) + 2 * U32 * want.abs()
        assert_close(t.t, want, err, "bias gradient")


@pytest.mark.parametrize("off", OFFS)
@pytest.mark.parametrize("M,K,f", SIZES)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_gated_grad(M, K, f, dt, off):
    gated_grad_case(M, K, f, dt, "silu", off)
    gated_grad_case(M, K, f, dt, "gelu", off, accumulate=True)


@pytest.mark.parametrize("off", OFFS)
@pytest.mark.parametrize("M,K,N", [(1500, 1021, 1031), (700, 2049, 1027)])
def test_odd_widths_that_are_copied(M, K, N, off):
    """Rows that do not start on 16 bytes are copied to a workspace first where that pays."""
    pad = (K + 7) // 8 * 8
    # at least the copies of q and x for the weight's gradient
    assert binding._dense_ws("ttt_linear_grad_ws_bytes", M, K, N, 1, 1, 0) > 2 * M * N + 2 * M * pad
    linear_case(M, K, N, BF16, F32, "silu", True, True, 0.5, off)
    gated_case(M, K, N, BF16, "gelu", True, off)
    linear_grad_case(M, K, N, BF16, BF16, "gelu", 1.0, off, accumulate=True)
    gated_grad_case(M, K, N, BF16, "silu", off)


@pytest.mark.parametrize("M,K,N", [(2048, 4096, 256), (40, 8192, 128), (1300, 72, 2056), (5000, 264, 64)])
def test_splits_of_k_and_long_sums(M, K, N):
    """Few tiles and a long k (its parts are summed apart and joined), and a weight's gradient over many rows."""
    linear_case(M, K, N, BF16, F32, None, True, True, 1.0, 0)
    linear_grad_case(M, K, N, BF16, BF16, "silu", 1.0, 0, accumulate=True)
    gated_case(M, K, N, BF16, "silu", False, 0)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("M,K,N", [(40, 2048, 320), (300, 520, 392), (1233, 1024, 512), (2100, 264, 2052), (1500, 1021, 1031),
                                   (19, 40, 2056)])
def test_tiles_of_each_side(M, K, N, dt):
    """Sizes between which the tile's side and the number of parts change, in both types and every form."""
    linear_case(M, K, N, dt, F32, "gelu", True, True, 0.5, 0)
    gated_case(M, K, N, dt, "silu", True, 0)
    linear_grad_case(M, K, N, dt, dt, "silu", 1.0, 0, accumulate=True)
    gated_grad_case(M, K, N, dt, "gelu", 0)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("M,K,N", [(3, 5, 7), (130, 72, 1365), (700, 513, 1027)])
def test_odd_widths_with_and_without_sums(M, K, N, dt):
    """The bias' sums come with the elementwise pass or not at all; the other gradients are the same bits."""
    g = torch.Generator().manual_seed(M + K + N)
    dy, pre, u = (make((M, N), dt, g).cuda() for _ in range(3))
    x, w, v = make((M, K), dt, g).cuda(), make((N, K), dt, g).cuda(), make((N, K), dt, g).cuda()
    a, b = (ttt.ttt_linear_grad(dy, x, w, act="silu", pre=pre, bias=k) for k in (True, False))
    assert b.dbias is None and torch.equal(a.dx, b.dx) and torch.equal(a.dw, b.dw)
    a, b = (ttt.ttt_gated_grad(dy, x, w, v, pre, u, bias=k) for k in (True, False))
    assert b.db_up is None and all(torch.equal(s, t) for s, t in zip(a[:3], b[:3]))
    # the last column's sums, next to which q has its zeros
    s = torch.sigmoid(pre.double())
    want = dy.double() * u.double() * s * (1 + pre.double() * (1 - s))
    err = (64 + 2 * (M + 3)) * U32 * want.abs().sum(0) + 64 * U32 * (dy.double() * u.double()).abs().sum(0)
    assert_close(a.db_gate, want.sum(0).cpu(), err.cpu(), "db_gate")


def test_rows_past_32_bits():
    """300000 rows of 8192: 2.4e9 results, the last ones 4.9 GB on. Rows are independent, so each must be what a call on
    it and its neighbours alone gives (the same kernel and tile: bit for bit), and the weight's gradient what its two
    halves give together."""
    M, K, N = 300000, 64, 8192
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((M, K), generator=g, device="cuda").to(BF16)
    w = (torch.randn((N, K), generator=g, device="cuda") / 8).to(BF16)
    y = ttt.ttt_linear(x, w, act="silu")
    for r in (0, 262143, 262144, M - 600):
        want = x[r:r + 600].double() @ w.double().T
        want = want * torch.sigmoid(want)
        err = 64 * U32 + half_step(BF16)
        assert bool(((y[r:r + 600].double() - want).abs() <= err * want.abs() + 1e-4).all()), r
    z, a, b = ttt.ttt_gated(x, w, w, act="relu", keep=True)
    assert torch.equal(a, b) and torch.equal(a[-1000:], ttt.ttt_linear(x[-1000:].contiguous(), w))
    assert not bool(torch.isnan(z[::4099]).any())
    del z, a, b
    got = ttt.ttt_linear_grad(y, x, w, bias=True)
    top = ttt.ttt_linear_grad(y[:150000], x[:150000], w)
    low = ttt.ttt_linear_grad(y[150000:], x[150000:], w)
    assert torch.equal(got.dx[:150000], top.dx) and torch.equal(got.dx[150000:], low.dx)
    both = top.dw.double() + low.dw.double()
    scale = both.abs().max()
    assert float((got.dw.double() - both).abs().max()) <= 3 * half_step(BF16) * float(scale)
    want = sum(part.double().sum(0) for part in y.split(50000))
    assert float((got.dbias.double() - want).abs().max()) <= 1e-5 * float(want.abs().max())


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own."""
    g = torch.Generator().manual_seed(6)
    x, w = make((1500, 512), BF16, g).cuda(), make((520, 512), BF16, g, 0.05).cuda()
    dy = [make((1500, 520), F32, g).cuda() for _ in range(2)]
    want = [ttt.ttt_linear_grad(d, x, w, bias=True) for d in dy]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in range(2)]
    for _ in range(10):
        for k, s in enumerate(streams):
            got[k].append(ttt.ttt_linear_grad(dy[k], x, w, bias=True, stream=s))
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            for a, b in zip(r, want[k]):
                assert torch.equal(a, b)


def test_gradients_against_differences():
    """Along a random direction of every input: (L(+h) - L(-h)) / 2h against the gradients' sum. In fp32 a loss of
    magnitude |L| is off by some 10^3 U of the terms' sum (about 2^-14 of its norm here) over 2h, and the third
    derivative adds h^2: with h = 2^-5 both stay below 2 % of the directional derivative's scale."""
    g = torch.Generator().manual_seed(5)
    M, K, f, N = 40, 48, 56, 32
    x, wg, wu, wd = (make(s, F32, g, k).cuda() for s, k in (((M, K), 1.0), ((f, K), K ** -0.5), ((f, K), K ** -0.5),
                                                            ((N, f), f ** -0.5)))
    bg, bu, bd = (make((n,), F32, g, 0.3).cuda() for n in (f, f, N))
    dy = make((M, N), F32, g).cuda()

    def loss(p):
        z = ttt.ttt_gated(p[0], p[1], p[2], p[3], p[4], act="gelu")
        return float((ttt.ttt_linear(z, p[5], p[6], act="silu", scale=0.5).double() * dy.double()).sum())

    at = [x, wg, wu, bg, bu, wd, bd]
    z, kg, ku = ttt.ttt_gated(*at[:5], act="gelu", keep=True)
    _, pre = ttt.ttt_linear(z, wd, bd, act="silu", scale=0.5, keep=True)
    lin = ttt.ttt_linear_grad(dy, z, wd, act="silu", pre=pre, scale=0.5, bias=True)
    gat = ttt.ttt_gated_grad(lin.dx, x, wg, wu, kg, ku, act="gelu", bias=True)
    grads = [gat.dx, gat.dw_gate, gat.dw_up, gat.db_gate, gat.db_up, lin.dw, lin.dbias]
    h = 2.0 ** -5
    for i, (p, d) in enumerate(zip(at, grads)):
        v = torch.randn(p.shape, generator=g).cuda()
        v /= v.norm()
        up, down = list(at), list(at)
        up[i], down[i] = p + h * v, p - h * v
        slope = (loss(up) - loss(down)) / (2 * h)
        want = float((d.double() * v.double()).sum())
        assert abs(slope - want) <= 0.02 * float(d.double().norm()), (i, slope, want)


def test_parts_not_asked_for():
    g = torch.Generator().manual_seed(9)
    x, w, dy = make((30, 64), BF16, g).cuda(), make((72, 64), BF16, g).cuda(), make((30, 72), BF16, g).cuda()
    full = ttt.ttt_linear_grad(dy, x, w, bias=True)
    a = ttt.ttt_linear_grad(dy, x, w, need_dx=False)
    b = ttt.ttt_linear_grad(dy, x, w, need_dw=False, bias=True)
    assert a.dx is None and a.dbias is None and torch.equal(a.dw, full.dw)
    assert b.dw is None and torch.equal(b.dx, full.dx) and torch.equal(b.dbias, full.dbias)
    wu, z = make((72, 64), BF16, g).cuda(), make((30, 72), BF16, g).cuda()
    full = ttt.ttt_gated_grad(dy, x, w, wu, z, dy)
    a = ttt.ttt_gated_grad(dy, x, w, wu, z, dy, need_dx=False, bias=True)
    assert a.dx is None and torch.equal(a.dw_up, full.dw_up) and full.db_up is None and a.db_up is not None


@pytest.mark.parametrize("dt", [F32, BF16])
def test_no_rows(dt):
    w, wu = torch.randn(24, 16, device="cuda").to(dt), torch.randn(24, 16, device="cuda").to(dt)
    x, dy = torch.empty((0, 16), device="cuda", dtype=dt), torch.empty((0, 24), device="cuda", dtype=dt)
    assert ttt.ttt_linear(x, w).shape == (0, 24) and ttt.ttt_gated(x, w, wu).shape == (0, 24)
    got = ttt.ttt_linear_grad(dy, x, w, bias=True)
    assert got.dx.shape == (0, 16) and not got.dw.any() and not got.dbias.any()
    got = ttt.ttt_gated_grad(dy, x, w, wu, dy, dy, bias=True)
    assert not got.dw_gate.any() and not got.dw_up.any() and not got.db_gate.any() and not got.db_up.any()
    dw, db = torch.ones((24, 16), device="cuda", dtype=dt), torch.ones((24,), device="cuda")
    ttt.ttt_linear_grad(dy, x, w, bias=True, dw=dw, dbias=db, accumulate=True)
    assert bool((dw == 1).all()) and bool((db == 1).all())


def test_infinities_and_nans_stay_in_their_rows():
    g = torch.Generator().manual_seed(3)
    for dt in (F32, BF16):
        for M in (3, 300):
            x, w, wu = make((M, 200), dt, g).cuda(), make((136, 200), dt, g).cuda(), make((136, 200), dt, g).cuda()
            clean = ttt.ttt_linear(x, w, act="silu"), ttt.ttt_gated(x, w, wu, act="relu")
            bad = x.clone()
            bad[1, 7], bad[2, 199] = float("nan"), float("inf")
            got = ttt.ttt_linear(bad, w, act="silu"), ttt.ttt_gated(bad, w, wu, act="relu")
            for a, b in zip(got, clean):
                assert bool(a[1].isnan().all()) and not bool(a[2].isfinite().all())
                assert torch.equal(a[0], b[0]) and torch.equal(a[3:], b[3:])


def test_large_arguments_of_the_activations():
    """a and a' at arguments whose exponentials and cubes leave fp32: their limits, no NaN."""
    p = torch.tensor([-3e38, -1e20, -1e4, -200.0, -90.0, 90.0, 200.0, 1e4, 1e20, 3e38])
    one = torch.ones((1, 1), device="cuda")
    for act in ("silu", "gelu", "relu"):
        y = ttt.ttt_linear(p[:, None].cuda(), one, act=act).cpu()[:, 0]
        assert torch.equal(y[5:], p[5:]) and bool((y[:5].abs() < 1e-30).all()), (act, y)
        got = ttt.ttt_linear_grad(torch.ones((10, 1), device="cuda"), torch.ones((10, 1), device="cuda"), one, act=act,
                                  pre=p[:, None].cuda())
        assert bool((got.dx.cpu()[5:, 0] == 1).all()) and bool((got.dx.cpu()[:5].abs() < 1e-30).all()), (act, got.dx)


@pytest.mark.parametrize("M,K,N", [(4, 512, 1000), (700, 264, 520), (1000, 77, 90)])
def test_same_bits_again_on_another_stream_and_in_replays(M, K, N):
    g = torch.Generator().manual_seed(2)
    x, w, wu = make((M, K), BF16, g).cuda(), make((N, K), BF16, g, 0.1).cuda(), make((N, K), BF16, g, 0.1).cuda()
    dy = make((M, N), BF16, g).cuda()

    def step():
        z, a, b = ttt.ttt_gated(x, w, wu, keep=True)
        y, pre = ttt.ttt_linear(x, w, act="gelu", residual=dy, keep=True)
        return [z, a, b, y, *ttt.ttt_linear_grad(dy, x, w, act="gelu", pre=pre, bias=True),
                *ttt.ttt_gated_grad(dy, x, w, wu, a, b, bias=True)]

    want = step()
    for a, b in zip(step(), want):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ttt.ttt_linear(x, w, stream=side)
    z = ttt.ttt_gated(x, w, wu, stream=side)
    d = ttt.ttt_linear_grad(dy, x, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ttt.ttt_linear(x, w)) and torch.equal(z, want[0])
    assert torch.equal(d.dw, ttt.ttt_linear_grad(dy, x, w).dw)
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for k in range(3):
        x.mul_(0.5)
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_refusals_on_the_device():
    x, w = torch.zeros((8, 32), device="cuda"), torch.zeros((16, 32), device="cuda")
    y = torch.zeros((8, 16), device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        ttt.ttt_linear(torch.zeros((32, 8), device="cuda").T, w)
    with pytest.raises(ValueError, match="must be torch.float32"):
        ttt.ttt_linear(x, w.bfloat16())
    with pytest.raises(ValueError, match="shape"):
        ttt.ttt_linear(x, w, torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError, match=r"\[out\]\[32\]"):
        ttt.ttt_linear(x, w.T.contiguous())
    with pytest.raises(ttt.TTTError, match="fp32 y"):
        ttt.ttt_linear(x, w, dtype=BF16)
    with pytest.raises(ttt.TTTError, match="overlaps"):
        ttt.ttt_linear(x, w, y=x.view(-1)[:128].view(8, 16))
    with pytest.raises(ttt.TTTError, match="finite"):
        ttt.ttt_linear(x, w, scale=float("inf"))
    with pytest.raises(ttt.TTTError, match="b_gate"):
        ttt.ttt_gated(x, w, w, b_gate=torch.zeros(16, device="cuda"))
    with pytest.raises(ValueError, match="pre must be given"):
        ttt.ttt_linear_grad(y, x, w, act="silu")
    with pytest.raises(ValueError, match="accumulate into"):
        ttt.ttt_linear_grad(y, x, w, accumulate=True)
    with pytest.raises(ttt.TTTError, match="overlaps"):
        ttt.ttt_linear_grad(y, x, w, dw=w)
    with pytest.raises(ValueError, match="act must be"):
        ttt.ttt_gated(x, w, w, act=None)

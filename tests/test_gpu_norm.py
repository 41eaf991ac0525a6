"""The norms around a block and their gradients against the formulas in 64 bits.

Bounds. With u = 2^-24, a row sum of d elements passes at most
N = 8 ceil(d / 8192) + 22 additions per element (a thread's own, six within
its wave, sixteen over the waves), so it is off by at most N u of the sum of
the terms' magnitudes. r = (S/d + eps)^-1/2 then is off by (N/2 + 4) u
relative. The longest chain of a gradient, r^2 m with m = r sum(g o) / d, holds
r three times and one more sum, and enters a last sum: 3 (N/2 + 4) + 2 N and a
few products, under (4 N + 40) u of the magnitudes. On top comes the rounding
of the result to its type. A gradient of a gain sums over the rows: the rows
of one workgroup (at least 256 of them share the rows) and the up to 32 rows it
takes at a time, then the workgroups in 128 slices, then the slices in seven
steps. The bound below counts the workgroups at their most, and 48 additions
besides, which also covers the up to 11 rows of a workgroup at these sizes.
"""
import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.block_util import U32, Guarded, assert_close, guarded, half_step, rms64

F, B = torch.float32, torch.bfloat16
TYPES = [(F, F, F), (F, B, B), (F, F, B), (B, B, B)]
EPS = 1e-6
gpu = pytest.mark.gpu


def chain(d):
    n = 8 * -(-d // 8192) + 22
    return (4 * n + 40) * U32


def inputs(rows, d, types, gate, seed=0, w=F, gains=True, nxt=True):
    g = torch.Generator().manual_seed(seed)
    h, y, x = types

    def r(shape, dt, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g) * std + mean).to(dt)

    return dict(
        h=r((rows, d), h, 2.0), y=r((rows, d), y, 0.5), w=r((d,), w, 0.2, 1.0) if gains else None,
        gate=None if gate == "none" else r((d,), w, 0.5) if gate == "channel" else r((rows, d), y, 0.5),
        w_next=r((d,), w, 0.2, 1.0) if gains and nxt else None, dh=r((rows, d), h, 0.1), dx=r((rows, d), x, 0.1))


def dev(v):
    return None if v is None else v.cuda()


def post64(p, alpha, beta, nxt):
    """(o, x, bound of o, bound of x) before rounding."""
    h, y = p["h"].double(), p["y"].double()
    c = chain(h.shape[-1])
    w = 1.0 if p["w"] is None else p["w"].double()
    a = 1.0 if p["gate"] is None else p["gate"].double()
    br = beta * a * w * y * rms64(y, EPS)
    o = alpha * h + br
    bo = c * ((alpha * h).abs() + br.abs())
    if not nxt:
        return o, None, bo, None
    wn = torch.ones(h.shape[-1]).double() if p["w_next"] is None else p["w_next"].double()
    r = rms64(o, EPS)
    norm = o.norm(dim=-1, keepdim=True).clamp_min(1e-300)
    bx = wn.abs() * r * (bo + o.abs() * (bo.norm(dim=-1, keepdim=True) / norm + c))
    return o, wn * o * r, bo, bx


def grads64(p, alpha, beta, use_dx, use_dh, parts):
    """Formulas and bounds: {name: (value, bound)}."""
    d = p["y"].shape[-1]
    c = chain(d)
    y = p["y"].double()
    w = torch.ones(d).double() if p["w"] is None else p["w"].double()
    a = torch.ones(1).double() if p["gate"] is None else p["gate"].double()
    do = p["dh"].double() if use_dh else torch.zeros_like(y)
    mag = do.abs()
    out = {}
    rows = y.shape[0]
    adds = (-(-rows // max(parts, 1)) + -(-parts // 16) + 16 + 32) * U32
    if use_dx:
        o, dx = p["h"].double(), p["dx"].double()
        wn = torch.ones(d).double() if p["w_next"] is None else p["w_next"].double()
        r = rms64(o, EPS)
        g = dx * wn
        do = do + r * (g - o * r * (g * o * r).mean(-1, keepdim=True))
        mag = mag + r * (g.abs() + o.abs() * r * (g * o * r).abs().mean(-1, keepdim=True))
        if p["w_next"] is not None:
            t = dx * o * r
            out["dw_next"] = (t.sum(0), (adds + c) * t.abs().sum(0))
    q = rms64(y, EPS)
    n = y * q
    pp, pm = beta * a * w * do, (beta * a * w).abs() * mag
    out["dy"] = (q * (pp - n * (pp * n).mean(-1, keepdim=True)),
                 2 * c * q * (pm + n.abs() * (pm * n.abs()).mean(-1, keepdim=True)))
    out["dh"] = (alpha * do, 2 * c * abs(alpha) * mag)
    if p["w"] is not None:
        out["dw"] = ((beta * a * n * do).sum(0), (adds + 2 * c) * ((beta * a * n).abs() * mag).sum(0))
    if p["gate"] is not None:
        t, tm = beta * w * n * do, (beta * w * n).abs() * mag
        out["dgate"] = (t, 2 * c * tm) if p["gate"].dim() == 2 else (t.sum(0), (adds + 2 * c) * tm.sum(0))
    return out


def parts_of(rows, d):
    from chunk_wise_weight_amd import binding
    return binding._norm_ws(rows, d) // (8 * d)


SIZES = [(1, 8), (5, 9), (257, 64), (33, 100), (1031, 256), (7, 257), (130, 511), (12, 520), (61, 1023), (700, 2560),
         (8193, 520), (3, 4097), (5, 8192), (2, 8200), (3, 9001), (1, 65536)]


@gpu
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("types", TYPES, ids=["fff", "fbb", "ffb", "bbb"])
@pytest.mark.parametrize("rows,d", SIZES)
def test_post_and_next(rows, d, types, gate):
    alpha, beta = 0.75, 1.5
    p = inputs(rows, d, types, gate, seed=d + rows, w=F if types[2] == F or d % 2 else B)
    o64, x64, bo, bx = post64(p, alpha, beta, True)
    v = {k: guarded(dev(t)) if t is not None else None for k, t in p.items()}
    o, x = Guarded((rows, d), types[0]), Guarded((rows, d), types[2], off=1)
    ttt.ttt_norm_post(v["h"], v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta, eps=EPS, w_next=v["w_next"],
                      o=o.t, x=x.t)
    torch.cuda.synchronize()
    o.check(), x.check()
    assert_close(o.t, o64, bo + half_step(types[0]) * (o64.abs() + bo), "o")
    assert_close(x.t, x64, bx + half_step(types[2]) * (x64.abs() + bx), "x")
    # the norm after the block alone, in place, gives the same o
    o2, none = ttt.ttt_norm_post(v["h"], v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta, eps=EPS, o=v["h"])
    assert none is None and o2 is v["h"] and torch.equal(o2, o.t)


@gpu
@pytest.mark.parametrize("types", TYPES, ids=["fff", "fbb", "ffb", "bbb"])
@pytest.mark.parametrize("rows,d", SIZES)
def test_pre_and_its_gradient(rows, d, types):
    p = inputs(rows, d, types, "none", seed=d, w=F)
    c = chain(d)
    h, w, dx = p["h"].double(), p["w_next"].double(), p["dx"].double()
    r = rms64(h, EPS)
    x = ttt.ttt_norm_pre(dev(p["h"]), dev(p["w_next"]), eps=EPS, dtype=types[2])
    ref = w * h * r
    assert x.dtype == types[2]
    assert_close(x, ref, (c + 2 * half_step(types[2])) * ref.abs(), "x")
    bare = ttt.ttt_norm_pre(dev(p["h"]), eps=EPS, dtype=types[2])  # without a gain
    assert_close(bare, h * r, (c + 2 * half_step(types[2])) * (h * r).abs(), "x without gain")
    g = dx * w
    gm = r * (g.abs() + h.abs() * r * (g * h * r).abs().mean(-1, keepdim=True))
    t = dx * h * r
    adds = (-(-rows // parts_of(rows, d)) + -(-parts_of(rows, d) // 16) + 48) * U32
    for with_in in (True, False):
        din = p["dh"].double() if with_in else torch.zeros_like(h)
        want = din + r * (g - h * r * (g * h * r).mean(-1, keepdim=True))
        bound = 2 * c * (gm + din.abs())
        dh, dw = ttt.ttt_norm_pre_grad(dev(p["dx"]), dev(p["h"]), dev(p["w_next"]), eps=EPS,
                                       dh_in=dev(p["dh"]) if with_in else None)
        assert_close(dh, want, bound + half_step(types[0]) * (want.abs() + bound), "dh")
        assert_close(dw, t.sum(0), (adds + c) * t.abs().sum(0), "dw")


@gpu
@pytest.mark.parametrize("use", ["both", "dx", "dh"])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("types", TYPES, ids=["fff", "fbb", "ffb", "bbb"])
@pytest.mark.parametrize("rows,d", SIZES)
def test_post_gradient(rows, d, types, gate, use):
    alpha, beta = 0.75, 1.5
    p = inputs(rows, d, types, gate, seed=3 * d + rows, w=F if types[2] == F or d % 2 else B)
    use_dx, use_dh = use != "dh", use != "dx"
    want = grads64(p, alpha, beta, use_dx, use_dh, parts_of(rows, d))
    v = {k: guarded(dev(t)) if t is not None else None for k, t in p.items()}
    dh, dy = Guarded((rows, d), types[0]), Guarded((rows, d), types[1], off=1)
    got = ttt.ttt_norm_post_grad(v["dh"] if use_dh else None, v["dx"] if use_dx else None, v["h"], v["y"], v["w"],
                                 gate=v["gate"], alpha=alpha, beta=beta, eps=EPS, w_next=v["w_next"], dh=dh.t, dy=dy.t)
    torch.cuda.synchronize()
    dh.check(), dy.check()
    have = {k: t for k, t in got._asdict().items() if t is not None}
    assert set(have) == set(want)
    for k, t in have.items():
        val, bound = want[k]
        assert_close(t, val, bound + half_step(t.dtype) * (val.abs() + bound), k)
    # in place (dh on dh_in, dy on y), and again: the same bits
    again = ttt.ttt_norm_post_grad(v["dh"] if use_dh else None, v["dx"] if use_dx else None, v["h"], v["y"], v["w"],
                                   gate=v["gate"], alpha=alpha, beta=beta, eps=EPS, w_next=v["w_next"],
                                   dh=v["dh"] if use_dh else None, dy=v["y"])
    for k, t in again._asdict().items():
        assert t is None or torch.equal(t, have[k]), k


@gpu
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("rows,d", [(33, 100), (130, 511), (700, 2560), (3, 9001)])
def test_without_gains(rows, d, gate):
    """No gain on either norm: ones in the formulas, and no gradients of them."""
    alpha, beta = 1.0, -0.5
    p = inputs(rows, d, (F, B, B), gate, seed=d, gains=False)
    o64, x64, bo, bx = post64(p, alpha, beta, True)
    v = {k: dev(t) for k, t in p.items()}
    o, x = ttt.ttt_norm_post(v["h"], v["y"], gate=v["gate"], alpha=alpha, beta=beta, eps=EPS, next_norm=True)
    assert_close(o, o64, bo + half_step(F) * (o64.abs() + bo), "o")
    assert_close(x, x64, bx + half_step(B) * (x64.abs() + bx), "x")
    want = grads64(p, alpha, beta, True, True, parts_of(rows, d))
    got = ttt.ttt_norm_post_grad(v["dh"], v["dx"], v["h"], v["y"], gate=v["gate"], alpha=alpha, beta=beta, eps=EPS)
    have = {k: t for k, t in got._asdict().items() if t is not None}
    assert set(have) == set(want) == {"dh", "dy"} | ({"dgate"} if gate != "none" else set())
    for k, t in have.items():
        val, bound = want[k]
        assert_close(t, val, bound + half_step(t.dtype) * (val.abs() + bound), k)
    dh, dw = ttt.ttt_norm_pre_grad(v["dx"], v["h"], eps=EPS)
    assert dw is None and dh.dtype == F


@gpu
def test_two_streams_at_once():
    """Calls that run at the same time keep to their own workspaces and outputs."""
    cases = []
    for k, (rows, d) in enumerate([(3000, 1024), (2500, 2560)]):
        p = inputs(rows, d, (F, B, B), "channel", seed=k)
        v = {n: dev(t) for n, t in p.items()}
        args = (v["dh"], v["dx"], v["h"], v["y"], v["w"], v["gate"])
        cases.append((args, v["w_next"], ttt.ttt_norm_post_grad(*args, w_next=v["w_next"])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for k, (args, wn, _) in enumerate(cases):
            got[k].append(ttt.ttt_norm_post_grad(*args, w_next=wn, stream=streams[k]))
    torch.cuda.synchronize()
    for k, (_, _, want) in enumerate(cases):
        for g in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(g, want))


@gpu
def test_gradients_against_autograd_and_differences():
    """The gradient along a random direction: formula by autograd in 64 bits, and central differences of the forward
    kernel in fp32. The difference's own error is that of the same difference in 64 bits plus the forward's rounding
    over the step."""
    rows, d, alpha, beta, step = 6, 136, 0.75, 1.5, 2.0 ** -6
    p = inputs(rows, d, (F, F, F), "token", seed=11)
    v = {k: dev(t) for k, t in p.items()}

    def forward64(q):
        o = alpha * q["h"] + beta * q["gate"] * q["w"] * q["y"] * rms64(q["y"], EPS)
        return o, q["w_next"] * o * rms64(o, EPS)

    names = ["h", "y", "w", "gate", "w_next"]
    q = {k: p[k].double().requires_grad_() for k in names}
    o, x = forward64(q)
    co, cx = p["dh"].double(), p["dx"].double()
    auto = dict(zip(names, torch.autograd.grad((o * co).sum() + (x * cx).sum(), [q[k] for k in names])))
    o32, _ = ttt.ttt_norm_post(v["h"], v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta, eps=EPS,
                               w_next=v["w_next"])
    got = ttt.ttt_norm_post_grad(v["dh"], v["dx"], o32, v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta,
                                 eps=EPS, w_next=v["w_next"])
    mine = {"h": got.dh, "y": got.dy, "w": got.dw, "gate": got.dgate, "w_next": got.dw_next}
    gen = torch.Generator().manual_seed(5)
    for k in names:
        # o32 is rounded (2^-24 of o), which moves the gradients by a like share; rows * d terms in dw
        scale = auto[k].abs().max()
        assert (mine[k].double().cpu() - auto[k]).abs().max() <= 64 * chain(d) * scale, k
        direction = torch.randn(p[k].shape, generator=gen)

        def loss(sign, kernel):
            t = dict(p)
            # the step in fp32, so that both sides take the very same one
            t[k] = p[k] + sign * step * direction
            if kernel:
                c = {n: dev(z) for n, z in t.items()}
                oo, xx = ttt.ttt_norm_post(c["h"], c["y"], c["w"], gate=c["gate"], alpha=alpha, beta=beta, eps=EPS,
                                           w_next=c["w_next"])
                oo, xx = oo.double().cpu(), xx.double().cpu()
            else:
                oo, xx = forward64({n: z.double() for n, z in t.items()})
            return float((oo * co).sum() + (xx * cx).sum()), float((oo * co).abs().sum() + (xx * cx).abs().sum())

        lp, mp = loss(1, True)
        lm, mm = loss(-1, True)
        e64 = (loss(1, False)[0] - loss(-1, False)[0]) / (2 * step)
        along = float((auto[k] * direction.double()).sum())
        diff = (lp - lm) / (2 * step)
        # inputs t[k] are rounded to fp32 alike on both sides; each output is off by the chain's bound
        noise = 4 * chain(d) * (mp + mm) / (2 * step)
        assert abs(diff - along) <= abs(e64 - along) + noise, (k, diff, along, noise)
        assert abs(along) > noise  # the test says something


@gpu
def test_rows_of_zeros_infinities_and_nan_stay_their_own():
    d = 520
    p = inputs(6, d, (F, F, F), "channel", seed=2)
    clean_o, clean_x = ttt.ttt_norm_post(dev(p["h"]), dev(p["y"]), dev(p["w"]), gate=dev(p["gate"]),
                                         w_next=dev(p["w_next"]))
    h, y = p["h"].clone(), p["y"].clone()
    h[1] = 0.0
    y[1] = 0.0
    y[3, 7] = float("nan")
    h[4, 100] = float("inf")
    o, x = ttt.ttt_norm_post(dev(h), dev(y), dev(p["w"]), gate=dev(p["gate"]), w_next=dev(p["w_next"]))
    assert bool((o[1] == 0).all()) and bool((x[1] == 0).all())  # eps keeps the empty row finite
    assert bool(o[3].isnan().all()) and bool(x[3].isnan().all())
    assert bool(o[4, 100].isinf()) and bool(x[4, 100].isnan()) and bool((x[4, :100] == 0).all())
    for r in (0, 2, 5):
        assert torch.equal(o[r], clean_o[r]) and torch.equal(x[r], clean_x[r])
    # gradients: the zero row's are those of the formula with r = eps^-1/2
    h[3], h[4], y[3] = p["h"][3], p["h"][4], p["y"][3]
    q = dict(p, h=h, y=y)
    want = grads64(q, 1.0, 1.0, True, True, parts_of(6, d))
    v = {k: dev(t) for k, t in q.items()}
    got = ttt.ttt_norm_post_grad(v["dh"], v["dx"], v["h"], v["y"], v["w"], gate=v["gate"], w_next=v["w_next"])
    for k, t in got._asdict().items():
        val, bound = want[k]
        assert_close(t, val, bound + half_step(t.dtype) * (val.abs() + bound), k)


@gpu
@pytest.mark.parametrize("shape", [(0, 64), (3, 0, 2560)])
def test_no_rows(shape):
    d = shape[-1]
    z = torch.empty(shape, device="cuda")
    w = torch.ones(d, device="cuda")
    assert ttt.ttt_norm_pre(z, w).shape == shape
    dh, dw = ttt.ttt_norm_pre_grad(z, z, w)
    assert dh.shape == shape and bool((dw == 0).all())
    o, x = ttt.ttt_norm_post(z, z, w, gate=w, w_next=w)
    assert o.shape == shape and x.shape == shape
    g = ttt.ttt_norm_post_grad(z, z, z, z, w, gate=w, w_next=w)
    for t in (g.dw, g.dgate, g.dw_next):
        assert bool((t == 0).all())


@gpu
def test_another_stream_and_graph_replays():
    p = inputs(300, 2560, (F, B, B), "channel", seed=9)
    v = {k: dev(t) for k, t in p.items()}

    def step(stream=None):
        o, x = ttt.ttt_norm_post(v["h"], v["y"], v["w"], gate=v["gate"], w_next=v["w_next"], stream=stream)
        return [o, x] + list(ttt.ttt_norm_post_grad(v["dh"], v["dx"], o, v["y"], v["w"], gate=v["gate"],
                                                    w_next=v["w_next"], stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in range(4):
        v["y"].copy_(dev(p["y"]) * (k + 1))
        eager = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out)), k


def test_refusals():
    """Argument errors, before any device work (CPU tensors and raw addresses: nothing here is read)."""
    z = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="device tensor"):
        ttt.ttt_norm_pre(z)
    with pytest.raises(TypeError):
        ttt.ttt_norm_pre([1.0])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ttt.ttt_norm_pre(z.double())
    with pytest.raises(ValueError, match="contiguous"):
        ttt.ttt_norm_pre(torch.zeros(64, 4).t())
    with pytest.raises(ValueError, match="dimension"):
        ttt.ttt_norm_pre(torch.zeros(()))
    with pytest.raises(ValueError, match="dh_in or dx"):
        ttt.ttt_norm_post_grad(None, None, None, z)
    with pytest.raises(ValueError, match="o must be given"):
        ttt.ttt_norm_post_grad(None, z, None, z)
    L = ttt.lib()
    F32, BF16 = 0, 1

    def pre(h=1 << 20, hdt=F32, w=None, wdt=F32, eps=1e-6, rows=4, d=64, x=1 << 24, xdt=F32):
        return L.ttt_norm_pre(h, hdt, w, wdt, eps, rows, d, x, xdt, None)

    assert pre(h=None) == -1 and pre(x=None) == -1
    assert pre(d=7) == -2 and pre(d=65537) == -2 and pre(rows=-1) == -2 and pre(rows=1 << 31) == -2
    assert pre(hdt=2) == -3 and pre(xdt=5) == -3 and pre(wdt=9) == -3
    assert pre(hdt=BF16, xdt=F32) == -3
    assert pre(eps=0.0) == -7 and pre(eps=float("nan")) == -7 and pre(eps=float("inf")) == -7
    assert pre(h=(1 << 20) + 2) == -7 and "aligned" in ttt.ttt_last_error()
    assert pre(x=1 << 20) == -7 and "overlaps" in ttt.ttt_last_error()
    assert pre(x=(1 << 20) + 512) == -7
    assert pre(w=(1 << 24) + 4) == -7

    def post(h=1 << 20, y=1 << 21, ydt=F32, gate=None, kind=0, alpha=1.0, beta=1.0, o=1 << 22, x=None, hdt=F32):
        return L.ttt_norm_post(h, hdt, y, ydt, None, gate, kind, None, F32, alpha, beta, 1e-6, 4, 64, o, x, F32, None)

    assert post(y=None) == -1 and post(o=None) == -1
    assert post(kind=1) == -1 and post(kind=2) == -1 and post(kind=3, gate=1 << 23) == -7
    assert post(alpha=float("nan")) == -7 and post(beta=float("inf")) == -7
    assert post(hdt=BF16) == -3
    assert post(o=1 << 21) == -7 and post(o=(1 << 20) + 256) == -7  # o may be h and nothing else
    assert post(x=1 << 22) == -7

    def grad(dh_in=1 << 20, dx=1 << 21, o=1 << 22, y=1 << 23, dh=1 << 24, dy=1 << 25, dw=1 << 26, ws=1 << 27,
             nws=1 << 20, gate=None, kind=0, dgate=None):
        return L.ttt_norm_post_grad(dh_in, dx, F32, o, F32, y, F32, None, gate, kind, None, F32, 1.0, 1.0, 1e-6, 4, 64,
                                    dh, dy, dw, dgate, None, ws, nws, None)

    assert grad(dh_in=None, dx=None) == -1 and grad(o=None) == -1 and grad(dy=None) == -1 and grad(ws=None) == -1
    assert grad(nws=16) == -2 and "workspace" in ttt.ttt_last_error()
    assert grad(ws=(1 << 27) + 4) == -7
    assert grad(kind=2, gate=1 << 28) == -1
    assert grad(dh=1 << 22) == -7 and grad(dy=1 << 20) == -7 and grad(ws=1 << 24) == -7
    assert L.ttt_norm_ws_bytes(4, 64, None) == -1


@gpu
def test_refusals_of_the_binding():
    h = torch.zeros(4, 64, device="cuda")
    b = h.bfloat16()
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        ttt.ttt_norm_pre(h, torch.ones(63, device="cuda"))
    with pytest.raises(ttt.TTTError):
        ttt.ttt_norm_pre(b, dtype=torch.float32)
    with pytest.raises(ttt.TTTError):
        ttt.ttt_norm_post(b, h)
    with pytest.raises(ValueError, match="gate"):
        ttt.ttt_norm_post(h, h.clone(), gate=torch.ones(4, 1, device="cuda"))
    with pytest.raises(ValueError, match="row dimension"):
        ttt.ttt_norm_post(w, w.clone(), gate=w)
    with pytest.raises(ValueError, match="one dtype"):
        ttt.ttt_norm_post(h, h.clone(), w, w_next=w.bfloat16())
    with pytest.raises(ValueError, match="gate must be"):
        ttt.ttt_norm_post(h, b, gate=h)
    with pytest.raises(ValueError, match="contiguous"):
        ttt.ttt_norm_post(h, torch.zeros(64, 4, device="cuda").t())
    with pytest.raises(ttt.TTTError, match="overlaps"):
        ttt.ttt_norm_pre(h, x=h)
    with pytest.raises(ttt.TTTError, match="d must be"):
        ttt.ttt_norm_pre(torch.zeros(4, 7, device="cuda"))
    for call in (lambda: ttt.ttt_norm_pre(h, dtype=torch.float16),
                 lambda: ttt.ttt_norm_post(h, h.clone(), next_norm=True, dtype=torch.float64)):
        with pytest.raises(ValueError, match="dtype must be"):
            call()


@gpu
def test_more_rows_than_a_grid_side_counts():
    """2^29 + 3 rows of 8: their threads, one per row of eight columns, pass 2^32 in eights of lanes."""
    rows, d = 2 ** 29 + 3, 8
    h = torch.ones((rows, d), dtype=B, device="cuda")
    h[-1] = torch.arange(1, 9, device="cuda").to(B)
    x = ttt.ttt_norm_pre(h, eps=EPS)
    want = ttt.ttt_norm_pre(h[-2:].clone(), eps=EPS)
    assert torch.equal(x[-2:], want)
    assert bool((x[:-1] == 1).all())


@gpu
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("types", TYPES, ids=["fff", "fbb", "ffb", "bbb"])
@pytest.mark.parametrize("d", [64, 511, 520, 1023, 2560, 8200])
def test_a_row_does_not_depend_on_how_many_there_are(d, types, gate):
    """The same bits in a batch long enough for two rows per workgroup, in a short one, and without the next norm."""
    rows, kw = 8195, dict(alpha=0.75, beta=1.5, eps=EPS)
    p = inputs(rows, d, types, gate, seed=d)
    v = {k: dev(t) for k, t in p.items()}
    o, x = ttt.ttt_norm_post(v["h"], v["y"], v["w"], gate=v["gate"], w_next=v["w_next"], dtype=types[2], **kw)
    first = ttt.ttt_norm_pre(v["h"], v["w_next"], eps=EPS, dtype=types[2])
    for lo, hi in ((0, 1), (4000, 4101), (rows - 2, rows)):
        h, y = v["h"][lo:hi].clone(), v["y"][lo:hi].clone()
        a = v["gate"][lo:hi].clone() if gate == "token" else v["gate"]
        o2, x2 = ttt.ttt_norm_post(h, y, v["w"], gate=a, w_next=v["w_next"], dtype=types[2], **kw)
        assert torch.equal(o2, o[lo:hi]) and torch.equal(x2, x[lo:hi])
        assert torch.equal(ttt.ttt_norm_pre(h, v["w_next"], eps=EPS, dtype=types[2]), first[lo:hi])
    assert torch.equal(ttt.ttt_norm_post(v["h"], v["y"], v["w"], gate=v["gate"], **kw)[0], o)


@gpu
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("types", TYPES, ids=["fff", "fbb", "ffb", "bbb"])
@pytest.mark.parametrize("rows,d", [(3, 8), (35, 100), (9, 511), (5, 2560), (3, 4097), (2, 8200), (2, 9001),
                                    (1, 65536)])
def test_elements_of_1e18(rows, d, types, gate):
    """The largest elements that are supported: rows whose sums of squares leave fp32 (from a width of about 340 on),
    and whose r^2 lies at the end of its range. The bounds are those of any other row."""
    alpha, beta = 0.75, 1.5
    p = inputs(rows, d, types, gate, seed=d, w=F if types[2] == F or d % 2 else B)
    gen = torch.Generator().manual_seed(d)
    for k in ("h", "y"):
        sign = torch.randint(0, 2, (rows, d), generator=gen) * 2.0 - 1.0
        p[k] = (sign * (0.5e18 + 0.49e18 * torch.rand((rows, d), generator=gen))).to(p[k].dtype)
    v = {k: dev(t) for k, t in p.items()}
    o64, x64, bo, bx = post64(p, alpha, beta, True)
    o, x = ttt.ttt_norm_post(v["h"], v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta, eps=EPS,
                             w_next=v["w_next"], dtype=types[2])
    assert_close(o, o64, bo + half_step(types[0]) * (o64.abs() + bo), "o")
    assert_close(x, x64, bx + half_step(types[2]) * (x64.abs() + bx), "x")
    want = grads64(p, alpha, beta, True, True, parts_of(rows, d))
    got = ttt.ttt_norm_post_grad(v["dh"], v["dx"], v["h"], v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta,
                                 eps=EPS, w_next=v["w_next"])
    for k, t in got._asdict().items():
        if t is not None:
            val, bound = want[k]
            assert_close(t, val, bound + half_step(t.dtype) * (val.abs() + bound), k)
    h, w, dx = p["h"].double(), p["w_next"].double(), p["dx"].double()
    r, c = rms64(h, EPS), chain(d)
    assert_close(ttt.ttt_norm_pre(v["h"], v["w_next"], eps=EPS, dtype=types[2]), w * h * r,
                 (c + 2 * half_step(types[2])) * (w * h * r).abs(), "first norm")
    g = dx * w
    want = p["dh"].double() * 2.0 ** -60 + r * (g - h * r * (g * h * r).mean(-1, keepdim=True))
    bound = 2 * c * (p["dh"].double().abs() * 2.0 ** -60 +
                     r * (g.abs() + h.abs() * r * (g * h * r).abs().mean(-1, keepdim=True)))
    # a residual path's gradient as small as this one's share
    dh, _ = ttt.ttt_norm_pre_grad(v["dx"], v["h"], v["w_next"], eps=EPS, dh_in=v["dh"] * 2.0 ** -60)
    assert_close(dh, want, bound + half_step(types[0]) * (want.abs() + bound), "dh")


@gpu
def test_an_output_of_another_type_is_refused_by_name():
    h = torch.zeros(4, 64, device="cuda")
    for dt in (torch.float64, torch.float16):
        x = h.to(dt)
        with pytest.raises(ValueError, match="x must be float32 or bfloat16"):
            ttt.ttt_norm_pre(h, x=x, dtype=dt)
        with pytest.raises(ValueError, match="x must be float32 or bfloat16"):
            ttt.ttt_norm_post(h, h.clone(), x=x, dtype=dt)
        with pytest.raises(ValueError, match="x must be float32 or bfloat16"):
            ttt.ttt_embed(h, torch.zeros(4, dtype=torch.int32, device="cuda"), x=x, dtype=dt)


def test_widths_past_32_bits_are_refused():
    """A width that a 32-bit int would hold the low bits of only (meta tensors: no memory behind them)."""
    wide = torch.empty((1, 2 ** 32 + 64), device="meta")
    for call in (lambda: ttt.ttt_norm_pre(wide), lambda: ttt.ttt_norm_post(wide, wide),
                 lambda: ttt.ttt_norm_pre_grad(wide, wide), lambda: ttt.ttt_norm_post_grad(wide, wide, wide, wide)):
        with pytest.raises(ValueError, match=r"2\^31"):
            call()


# Workgroups of a gradient launch take rows in steps. Sizes where every form takes several: narrow rows side by side,
# ragged rows, rows of more than 512 threads, and rows too wide for registers; the last step not full. (8195, 1023) is
# also the forward with two ragged rows per workgroup, and an odd number of them.
STEPS = [(40000, 64), (9001, 256), (5003, 511), (8195, 1023), (601, 4097), (600, 8192), (600, 8200), (601, 9001)]


@gpu
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("types", TYPES, ids=["fff", "fbb", "ffb", "bbb"])
@pytest.mark.parametrize("rows,d", STEPS)
def test_gradients_of_several_steps(rows, d, types, gate):
    """Bounds as above, the sums over the rows counted at their longest: a launch has 256 workgroups at least, each of
    which takes ceil(rows / 256) rows at most one after another and joins 32 rows side by side at most; of the at most
    2048 partial sums 16 follow one another, and seven steps join the slices: under ceil(rows / 256) + 16 + 48."""
    alpha, beta = 0.75, 1.5
    p = inputs(rows, d, types, gate, seed=rows, w=F if types[2] == F or d % 2 else B)
    v = {k: dev(t) for k, t in p.items()}
    with torch.device("cuda"):  # the formulas in 64 bits, computed there for speed
        o64, x64, bo, bx = post64(v, alpha, beta, True)
        want = grads64(v, alpha, beta, True, True, 256)
    o, x = ttt.ttt_norm_post(v["h"], v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta, eps=EPS,
                             w_next=v["w_next"], dtype=types[2])
    assert_close(o, o64.cpu(), (bo + half_step(types[0]) * (o64.abs() + bo)).cpu(), "o")
    assert_close(x, x64.cpu(), (bx + half_step(types[2]) * (x64.abs() + bx)).cpu(), "x")
    keep = [v[k].clone() for k in ("dx", "h")]
    dh, dy = Guarded((rows, d), types[0]), Guarded((rows, d), types[1], off=1)
    got = ttt.ttt_norm_post_grad(v["dh"], v["dx"], v["h"], v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta,
                                 eps=EPS, w_next=v["w_next"], dh=dh.t, dy=dy.t)
    torch.cuda.synchronize()
    dh.check(), dy.check()
    have = {k: t for k, t in got._asdict().items() if t is not None}
    assert set(have) == set(want)
    for k, t in have.items():
        val, bound = want[k]
        assert_close(t, val.cpu(), (bound + half_step(t.dtype) * (val.abs() + bound)).cpu(), k)
    # without the residual path's gradient, and without the next norm's: the same forms with fewer inputs
    with torch.device("cuda"):
        some = [(None, v["dx"], grads64(v, alpha, beta, True, False, 256)),
                (v["dh"], None, grads64(v, alpha, beta, False, True, 256))]
    for dh_in, dx, want in some:
        part = ttt.ttt_norm_post_grad(dh_in, dx, v["h"], v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta,
                                      eps=EPS, w_next=v["w_next"])
        for k, t in part._asdict().items():
            if t is not None:
                val, bound = want[k]
                assert_close(t, val.cpu(), (bound + half_step(t.dtype) * (val.abs() + bound)).cpu(), k)
    # in place: the same bits, and the inputs as they were
    again = ttt.ttt_norm_post_grad(v["dh"], v["dx"], v["h"], v["y"], v["w"], gate=v["gate"], alpha=alpha, beta=beta,
                                   eps=EPS, w_next=v["w_next"], dh=v["dh"], dy=v["y"])
    assert again.dh is v["dh"] and again.dy is v["y"]
    for k, t in have.items():
        assert torch.equal(getattr(again, k), t), k
    assert torch.equal(v["dx"], keep[0]) and torch.equal(v["h"], keep[1])


@gpu
@pytest.mark.parametrize("types", TYPES, ids=["fff", "fbb", "ffb", "bbb"])
@pytest.mark.parametrize("rows,d", STEPS)
def test_first_norm_gradient_of_several_steps(rows, d, types):
    p = inputs(rows, d, types, "none", seed=rows + 1, w=F)
    v = {k: dev(t) for k, t in p.items()}
    c, adds = chain(d), (-(-rows // 256) + 16 + 48) * U32
    h, w, dx, din = (v[k].double() for k in ("h", "w_next", "dx", "dh"))
    r = rms64(h, EPS)
    g = dx * w
    want = din + r * (g - h * r * (g * h * r).mean(-1, keepdim=True))
    bound = 2 * c * (din.abs() + r * (g.abs() + h.abs() * r * (g * h * r).abs().mean(-1, keepdim=True)))
    t = dx * h * r
    dh, dw = ttt.ttt_norm_pre_grad(v["dx"], v["h"], v["w_next"], eps=EPS, dh_in=v["dh"])
    assert_close(dh, want.cpu(), (bound + half_step(types[0]) * (want.abs() + bound)).cpu(), "dh")
    assert_close(dw, t.sum(0).cpu(), ((adds + c) * t.abs().sum(0)).cpu(), "dw")
    again, dw2 = ttt.ttt_norm_pre_grad(v["dx"], v["h"], v["w_next"], eps=EPS, dh_in=v["dh"], dh=v["dh"])
    assert again is v["dh"] and torch.equal(again, dh) and torch.equal(dw2, dw)
    ref = w * h * r
    x = ttt.ttt_norm_pre(v["h"], v["w_next"], eps=EPS, dtype=types[2])
    assert_close(x, ref.cpu(), ((c + 2 * half_step(types[2])) * ref.abs()).cpu(), "x")

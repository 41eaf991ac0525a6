"""The global gradient norm and clipping against the formulas in 64 bits.

Bounds. Squares of fp32 values are exact in fp64 and the sums are off by at
most 2^20 steps of 2^-53 here, far below fp32, so the norm is off by its one
rounding, u = 2^-24 (with a hair for the sum). The factor tau / N is rounded
once, the product once in fp32 and once to its type.
"""
import ctypes
import math

import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.block_util import U32, assert_close, half_step

F, B16 = torch.float32, torch.bfloat16
gpu = pytest.mark.gpu


def make(sizes, dtypes, std=1e-3, seed=0, gap=1):
    """Tensors of the given sizes, each of its type's buffer, `gap` marked elements apart (None: touching)."""
    g = torch.Generator().manual_seed(seed)
    bufs, views = {}, []
    for dt in set(dtypes):
        n = sum(s + (gap or 0) for s, t in zip(sizes, dtypes) if t == dt) + 1
        bufs[dt] = torch.full((n,), 77.0, dtype=dt, device="cuda")
    at = {dt: 1 for dt in bufs}
    for s, dt in zip(sizes, dtypes):
        v = bufs[dt][at[dt]:at[dt] + s]
        v.copy_((torch.randn(s, generator=g) * std).to(dt))
        views.append(v)
        at[dt] += s + (gap or 0)
    return bufs, views


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


CASES = {
    "one": ([1], [F]),
    "small": ([3, 0, 2560, 1, 17, 2048, 2049], [F, B16, F, B16, F, F, B16]),
    "many": ([(i * 37) % 301 for i in range(700)], [F if i % 3 else B16 for i in range(700)]),
    "large": ([5_000_001, 8, 3_000_007, 2048 * 2048], [F, F, B16, B16]),
}


@gpu
@pytest.mark.parametrize("gap", [None, 1, 8])
@pytest.mark.parametrize("name", CASES)
def test_norm_and_clipping(name, gap):
    sizes, dtypes = CASES[name]
    bufs, g = make(sizes, dtypes, gap=gap)
    n64 = norm64(g)
    before = {dt: b.clone() for dt, b in bufs.items()}
    n = ttt.ttt_grad_norm(g)
    assert n.shape == (1,) and n.dtype == F
    assert abs(float(n) - n64) <= 1.01 * U32 * n64
    for tau in (0.3 * n64, 2.0 * n64):
        c = min(1.0, float(torch.tensor(tau, dtype=F)) / n64)
        # into a copy: every element written, the gradients left alone
        obufs, out = make(sizes, dtypes, seed=1, gap=gap)
        assert float(ttt.ttt_clip_grads(g, tau, out=out)) == float(n)
        for b, a in zip(g, out):
            ref = b.double().cpu() * c
            assert_close(a, ref, (2.02 * U32 + 1.01 * half_step(a.dtype)) * ref.abs(), "out")
        for dt in bufs:
            assert torch.equal(bufs[dt], before[dt])
        if gap:  # the marks between are as they were
            for dt, b in obufs.items():
                assert int((b == 77.0).sum()) == int((bufs[dt] == 77.0).sum())
        # in place, the same bits
        ibufs, ing = make(sizes, dtypes, gap=gap)
        assert float(ttt.ttt_clip_grads(ing, tau)) == float(n)
        for a, b in zip(ing, out):
            assert torch.equal(a, b)
        if tau > n64:
            for dt in bufs:
                assert torch.equal(ibufs[dt], before[dt])


@gpu
def test_same_bits_again_and_in_a_list_twice():
    _, g = make(*CASES["large"], gap=1)
    first = ttt.ttt_grad_norm(g)
    for _ in range(3):
        assert torch.equal(ttt.ttt_grad_norm(g), first)
    twice = ttt.ttt_grad_norm(g + g)
    assert abs(float(twice) - math.sqrt(2) * norm64(g)) <= 1.01 * U32 * float(twice)
    with pytest.raises(ttt.TTTError, match="overlaps"):
        ttt.ttt_clip_grads(g + g[:1], 1.0)
    with pytest.raises(ttt.TTTError, match="overlaps"):
        ttt.ttt_clip_grads(g[:1], 1.0, out=[shifted(g[0])])


def shifted(t):
    """A view of t's buffer that lies one element further."""
    return torch.as_strided(t, t.shape, t.stride(), t.storage_offset() + 1)


@gpu
@pytest.mark.parametrize("std", [1e-30, 1e18, 3e37])
def test_squares_that_leave_fp32(std):
    _, g = make([5000, 77], [F, B16], std=std)
    n64 = norm64(g)
    n = float(ttt.ttt_grad_norm(g))
    assert (abs(n - n64) <= 1.01 * U32 * n64) if n64 < 3.4e38 else n == math.inf
    tau = 0.25 * min(n64, 1e38)
    out = [torch.empty_like(t) for t in g]
    ttt.ttt_clip_grads(g, tau, out=out)
    c = float(torch.tensor(tau, dtype=F)) / n64
    for a, b in zip(out, g):
        ref = b.double().cpu() * c
        # results near the bottom of the type lose bits to its smallest step
        assert_close(a, ref, (2.02 * U32 + 1.01 * half_step(a.dtype)) * ref.abs() + 2.0 ** -133, "out")


@gpu
def test_factor_below_fp32():
    """tau / N past the smallest fp32 number, with results well inside it."""
    _, g = make([5000, 77], [F, B16], std=1e30)
    n64 = norm64(g)
    tau = 1e-10
    out = [torch.empty_like(t) for t in g]
    ttt.ttt_clip_grads(g, tau, out=out)
    c = float(torch.tensor(tau, dtype=F)) / n64
    assert c < 1e-41
    for a, b in zip(out, g):
        ref = b.double().cpu() * c
        assert_close(a, ref, (2.02 * U32 + 1.01 * half_step(a.dtype)) * ref.abs(), "out")


@gpu
def test_more_than_the_caches_hold_unaligned():
    """600 MB, which is read and written past the caches, from odd addresses."""
    n = 300_000_001
    buf = torch.full((n + 3,), 77.0, dtype=B16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    g = buf[1:1 + n]
    g.copy_(torch.randn(n, generator=gen, device="cuda"))
    n64 = float(torch.linalg.vector_norm(g, dtype=torch.float64))
    out = torch.full((n + 6,), 77.0, dtype=B16, device="cuda")
    norm = ttt.ttt_clip_grads([g], 0.5 * n64, out=[out[3:3 + n]])
    assert abs(float(norm) - n64) <= 1.01 * U32 * n64
    # the factor is a half but for its rounding, so a value may end one step off where it lies between two steps
    ref = (g.float() * 0.5)
    assert bool(((out[3:3 + n].float() - ref).abs() <= ref.abs() * 2.0 ** -7).all())
    assert bool((out[:3] == 77).all()) and bool((out[3 + n:] == 77).all())
    assert bool((buf[:1] == 77).all()) and bool((buf[1 + n:] == 77).all())


@gpu
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(bad):
    _, g = make([5000, 77], [F, B16])
    g[0][4321] = bad
    keep = [t.clone() for t in g]
    n = ttt.ttt_clip_grads(g, 1e-3)
    assert not bool(n.isfinite())
    for a, b in zip(g, keep):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = [torch.zeros_like(t) for t in g]
    ttt.ttt_clip_grads(g, 1e-3, out=out)
    for a, b in zip(out, keep):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@gpu
def test_empty_lists_and_infinite_threshold():
    assert float(ttt.ttt_grad_norm([])) == 0.0
    assert float(ttt.ttt_clip_grads([], 1.0)) == 0.0
    z = torch.empty(0, device="cuda")
    assert float(ttt.ttt_clip_grads([z, z], 1.0)) == 0.0
    _, g = make([100], [F])
    keep = g[0].clone()
    ttt.ttt_clip_grads(g, math.inf)
    assert torch.equal(g[0], keep)
    zero = [torch.zeros(9, device="cuda")]
    assert float(ttt.ttt_clip_grads(zero, 1e-30)) == 0.0 and bool((zero[0] == 0).all())


@gpu
def test_another_stream_and_graph_replays():
    sizes, dtypes = CASES["many"]
    _, g = make(sizes, dtypes)
    out = [torch.empty_like(t) for t in g]
    n64 = norm64(g)
    want_n = ttt.ttt_clip_grads(g, 0.5 * n64, out=out).clone()
    want = [t.clone() for t in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = [torch.empty_like(t) for t in g]
    side.wait_stream(torch.cuda.current_stream())
    n = ttt.ttt_clip_grads(g, 0.5 * n64, out=out2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n, want_n) and all(torch.equal(a, b) for a, b in zip(want, out2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gn = ttt.ttt_clip_grads(g, 0.5 * n64, out=out2)
    for k in range(4):
        for t in g:
            t.mul_(1.5)
        eager_n = ttt.ttt_clip_grads(g, 0.5 * n64, out=out)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gn, eager_n) and all(torch.equal(a, b) for a, b in zip(out, out2)), k


def test_refusals():
    z = torch.zeros(4)
    with pytest.raises(ValueError, match="device"):
        ttt.ttt_grad_norm([z])
    with pytest.raises(TypeError):
        ttt.ttt_grad_norm([1.0])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ttt.ttt_grad_norm([z.half()])
    with pytest.raises(ValueError, match="contiguous"):
        ttt.ttt_grad_norm([torch.zeros(4, 4).t()])
    L = ttt.lib()
    BASE = 1 << 30

    def call(ptrs=(BASE, BASE + 4096), sizes=(16, 16), dts=(0, 1), n=None, tau=1.0, out=None, norm=1 << 20,
             ws=1 << 21, nws=1 << 20):
        p = (ctypes.c_void_p * len(ptrs))(*ptrs)
        s = (ctypes.c_int64 * len(sizes))(*sizes)
        d = (ctypes.c_int32 * len(dts))(*dts)
        o = None if out is None else (ctypes.c_void_p * len(out))(*out)
        n = len(ptrs) if n is None else n
        return L.ttt_clip_grads(p, s, d, n, tau, o, norm, ws, nws, None)

    assert L.ttt_clip_grads(None, None, None, 1, 1.0, None, 1 << 20, 1 << 21, 1 << 20, None) == -1
    assert call(n=-1) == -2 and call(n=(1 << 20) + 1) == -2
    assert call(norm=None) == -1 and call(ws=None) == -1 and call(ptrs=(BASE, None)) == -1
    assert call(out=(BASE, None)) == -1
    assert call(nws=64) == -2 and call(sizes=(16, -1)) == -2 and call(sizes=(1 << 40, 1)) == -2
    assert call(dts=(0, 7)) == -3
    assert call(tau=0.0) == -7 and call(tau=-1.0) == -7 and call(tau=float("nan")) == -7
    assert call(ptrs=(BASE + 2, BASE + 4096)) == -7 and call(ptrs=(BASE, BASE + 4097)) == -7
    assert call(norm=(1 << 20) + 2) == -7 and call(ws=(1 << 21) + 8) == -7
    assert call(out=(BASE + 4, BASE + 4096)) == -7  # one element further than its gradient
    assert call(out=(BASE + 8192, BASE + 8192)) == -7
    assert call(ptrs=(BASE, BASE)) == -7
    assert call(norm=BASE + 8) == -7 and call(ws=BASE + 4096) == -7 and call(norm=1 << 21) == -7
    n = ctypes.c_size_t()
    assert L.ttt_grad_ws_bytes(-1, ctypes.byref(n)) == -2 and L.ttt_grad_ws_bytes(1, None) == -1


@gpu
def test_refusals_of_the_binding():
    g = [torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda", dtype=B16)]
    with pytest.raises(ValueError, match="one tensor per"):
        ttt.ttt_clip_grads(g, 1.0, out=g[:1])
    with pytest.raises(ValueError, match="dtypes and sizes"):
        ttt.ttt_clip_grads(g, 1.0, out=[g[1].clone(), g[0].clone()])
    with pytest.raises(ValueError, match="contiguous"):
        ttt.ttt_clip_grads([torch.zeros(8, 8, device="cuda").t()], 1.0)
    with pytest.raises(ValueError, match="shape"):
        ttt.ttt_grad_norm(g, norm=torch.zeros((), device="cuda"))


def at_a_tie():
    """Two tensors whose norm tells the order of its sum. The first one's squares add to 1 + 2^-23 + 5 s, s = 2^-52 the
    step of a sum near 1; a square of the second is b^2 = s / 20, 252 of them 12.6 s. Added apart and then at once they
    move the sum by 13 s; added by fours, eights, ... 128 (a wave whose first lane holds the first tensor) by
    0 + 0 + 1 + 2 + 3 + 6 = 12. The root of the sum with 12 s is the tie 1 + 2^-24, which fp32 rounds to 1, with 13 s
    it lies past it."""
    first = torch.tensor([1.0, 2.0 ** -12, 2.0 ** -12, math.sqrt(5.0) * 2.0 ** -26])
    return first, torch.full((252,), math.sqrt(0.05) * 2.0 ** -26)


@gpu
@pytest.mark.parametrize("gap,want", [(0, 1.0), (1, 1.0 + 2.0 ** -23), (1000, 1.0 + 2.0 ** -23)])
def test_the_norm_does_not_depend_on_where_outputs_lie(gap, want):
    """Gradients that adjoin in memory are summed as one, others apart, whichever call it is and wherever it writes."""
    first, second = at_a_tie()
    buf = torch.full((4 + gap + 252,), 77.0, device="cuda")
    g = [buf[:4], buf[4 + gap:]]
    g[0].copy_(first), g[1].copy_(second)
    norms = [float(ttt.ttt_grad_norm(g))]
    for apart in (0, 3):
        obuf = torch.full((4 + apart + 252,), 77.0, device="cuda")
        out = [obuf[:4], obuf[4 + apart:]]
        norms.append(float(ttt.ttt_clip_grads(g, 0.5, out=out)))
        # the factor is 1/2 (1 - 2^-24 or so), rounded once, as is each product
        for a, b in zip(out, (first, second)):
            assert_close(a, b.double() * 0.5, 4 * U32 * b.double(), "out")
        assert bool((obuf[4:4 + apart] == 77).all())
        norms.append(float(ttt.ttt_clip_grads(g, 0.5, out=[g[0].clone(), out[1]])))
    norms.append(float(ttt.ttt_clip_grads(g, 2.0)))
    assert norms == [want] * len(norms)

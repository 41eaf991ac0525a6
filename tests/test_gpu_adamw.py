"""The AdamW step over many tensors: fp32 moments against the formula in 64 bits, 8-bit ones against its codes, worked
out here from the definition in include/ttt.h with whole numbers and fp64."""
import math

import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.block_util import U32, assert_close, half_step

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HYPER = dict(betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


def step64(w, g, m, v, step, lr, betas, eps, weight_decay, factor=1.0):
    b1, b2 = betas
    g = g.double() * factor
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    upd = lr * (m / (1 - b1 ** step)) / (torch.sqrt(v / (1 - b2 ** step)) + eps)
    return w.double() * (1 - lr * weight_decay) - upd, m, v, upd


# a scalar, the sides of vectors, blocks and chunks, a matrix
SHAPES = [(1,), (3,), (255,), (256,), (257,), (5, 0), (4096,), (4097,), (33, 125), (64, 200), (2,), (100000,)]


def lists(shapes, wdt, gdt, seed, gap):
    """Views of flat buffers (gap 0: back to back) and the buffers, which hold marks between the views."""
    g = torch.Generator().manual_seed(seed)
    sizes = [math.prod(s) for s in shapes]
    out = []
    for dt, std in ((wdt, 0.5), (gdt, 1e-2), (F32, 1e-3), (F32, 1e-2)):
        flat = torch.full((sum(sizes) + gap * len(sizes) + gap,), 77.0, dtype=dt, device="cuda")
        at, views = gap, []
        for n, s in zip(sizes, shapes):
            views.append(flat[at:at + n].view(s))
            views[-1].copy_((torch.randn(s, generator=g) * std).to(dt))
            at += n + gap
        out.append((flat, views))
    out[3][1][:] = [v.square_() for v in out[3][1]]
    return out


@pytest.mark.parametrize("gap", [0, 3])
@pytest.mark.parametrize("wdt,gdt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("clip", [None, 0.5, 2.0])
def test_moments_in_fp32(wdt, gdt, gap, clip):
    """m and v: three roundings of their terms. w: the shrinking is one, and of the step's quotient each factor is a few
    roundings off, 16 together; the result is rounded to its type."""
    (fw, w), (fg, g), (fm, m), (fv, v) = lists(SHAPES, wdt, gdt, 3, gap)
    old = [[t.clone() for t in ts] for ts in (w, m, v)]
    copies = [torch.zeros(s, dtype=BF16, device="cuda") for s in SHAPES]
    norm, kw, factor = None, {}, 1.0
    if clip:
        norm = ttt.ttt_grad_norm(g)
        tau = clip * float(norm)
        kw = dict(norm=norm, tau=tau)
        factor = min(1.0, tau / float(norm.double()))
    ttt.ttt_adamw(w, g, m, v, 7, 1e-2, copies=copies, **kw, **HYPER)
    for i in range(len(SHAPES)):
        ww, wm, wv, upd = (t.cpu() for t in step64(old[0][i], g[i], old[1][i], old[2][i], 7, 1e-2, factor=factor, **HYPER))
        gd, om, ov = g[i].double().cpu() * factor, old[1][i].double().cpu(), old[2][i].double().cpu()
        assert_close(m[i], wm, 4 * U32 * (0.9 * om.abs() + 0.1 * gd.abs()), "m")
        assert_close(v[i], wv, 6 * U32 * (ov + 1e-3 * gd * gd), "v")
        em = 4 * U32 * (0.9 * om.abs() + 0.1 * gd.abs()) / wm.abs().clamp(min=1e-300)
        err = 2 * U32 * ww.abs() + U32 * old[0][i].double().cpu().abs() + upd.abs() * (16 * U32 + em)
        assert_close(w[i], ww, err + half_step(wdt) * (ww.abs() + err), "w")
        assert_close(copies[i], ww, err + half_step(BF16) * (ww.abs() + err), "copy")
    for flat, views in ((fw, w), (fg, g), (fm, m), (fv, v)):
        touched = torch.zeros(flat.shape, dtype=torch.bool, device="cuda")
        for t in views:
            if t.numel():
                touched[t.storage_offset():t.storage_offset() + t.numel()] = True
        assert bool((flat[~touched] == 77.0).all()), "written between the tensors"


def test_some_steps_from_nothing():
    """Twenty steps on a quadratic, each against 64 bits on what it was given."""
    g = torch.Generator().manual_seed(1)
    w = torch.randn(1000, generator=g).cuda()
    m, v = torch.zeros_like(w), torch.zeros_like(w)
    for t in range(1, 21):
        grad = 0.3 * w
        ow, om, ov = w.clone(), m.clone(), v.clone()
        ttt.ttt_adamw([w], [grad], [m], [v], t, 0.05, betas=(0.8, 0.9), eps=1e-6, weight_decay=0.0)
        ww, wm, wv, upd = step64(ow, grad, om, ov, t, 0.05, (0.8, 0.9), 1e-6, 0.0)
        e = 4 * U32 * (0.8 * om.double().abs() + 0.2 * grad.double().abs()) / wm.abs().clamp(min=1e-300)
        err = 2 * U32 * ww.abs() + U32 * ow.double().abs() + upd.abs() * (16 * U32 + e)
        assert_close(w, ww.cpu(), err.cpu(), f"step {t}")


# ---- 8 bits ----

def mix(h):
    h = ((h ^ (h >> 16)) * 0x6C8E9CF5) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0x51ED2701) & 0xFFFFFFFF
    return h ^ (h >> 16)


GOLDEN = 0x9E3779B1


def bits_of(seed, step, tensor, n):
    key = mix((seed + GOLDEN * mix(step & 0xFFFFFFFF)) & 0xFFFFFFFF)
    key = mix((key + GOLDEN * (tensor + 1)) & 0xFFFFFFFF)
    e = np.arange(n, dtype=np.uint64)
    return mix((np.uint64(key) + e * np.uint64(GOLDEN)) & np.uint64(0xFFFFFFFF)).astype(np.int64)


def pattern(k):
    return (np.maximum(k, 0).astype(np.uint32) << np.uint32(20)).view(np.float32)


def values(codes, tops, most):
    """codes [n], tops [blocks] -> float32."""
    c = codes.astype(np.int64)
    top = np.repeat(tops.astype(np.int64), 256)[:c.size]
    k = c & most
    v = np.where(k > 0, pattern(top - most + k), np.float32(0))
    return np.where(c >= 128, -v, v).astype(np.float32) if most == 127 else v.astype(np.float32)


def encode(x, r, most):
    """x float32 -> (codes, tops)."""
    n = x.size
    mag = np.abs(x).view(np.uint32).astype(np.int64)
    padded = np.concatenate([mag, np.zeros(-n % 256, np.int64)]).reshape(-1, 256)
    tops = (padded.max(1) + 0xFFFFF) >> 20
    top = np.repeat(tops, 256)[:n]
    c = ((mag + 16 * r) >> 20) - top + most
    least = pattern(top - most + 1)
    share = ((r + 0.5) / 65536).astype(np.float32)
    low = (np.abs(x) >= share * least).astype(np.int64) if most == 127 else np.ones(n, np.int64)
    c = np.where(mag == 0, 0, np.where(c < 1, low, c))
    if most == 127:
        c = c + 128 * ((x < 0) & (c > 0))
    return c.astype(np.uint8), tops.astype(np.int16)


def state8(shapes, seed, spread):
    """Codes and tops of random moments whose magnitudes run over many octaves."""
    rng = np.random.default_rng(seed)
    ms, vs, tops = [], [], []
    for s in shapes:
        n = math.prod(s)
        m = (rng.standard_normal(n) * 2.0 ** rng.uniform(-spread, 0, n)).astype(np.float32)
        v = np.square(rng.standard_normal(n) * 2.0 ** rng.uniform(-spread, 0, n)).astype(np.float32)
        cm, tm = encode(m, np.zeros(n, np.int64), 127)
        cv, tv = encode(v, np.zeros(n, np.int64), 255)
        ms.append(torch.from_numpy(cm).view(s).cuda())
        vs.append(torch.from_numpy(cv).view(s).cuda())
        tops.append(torch.from_numpy(np.stack([tm, tv]).reshape(2, -1)).cuda())
    return ms, vs, tops


@pytest.mark.parametrize("wdt,gdt", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("spread", [0, 30])
@pytest.mark.parametrize("clip", [False, True])
def test_moments_in_8_bits(wdt, gdt, spread, clip):
    (_, w), (_, g), _, _ = lists(SHAPES, wdt, gdt, 5, 3)
    if spread:
        for t in g:
            t.mul_(torch.exp2(-torch.rand(t.shape, device="cuda") * spread))
    ms, vs, tops = state8(SHAPES, 7, spread)
    before = [[t.cpu().numpy().copy() for t in ts] for ts in (ms, vs, tops)]
    ow = [t.clone() for t in w]
    kw, factor = {}, 1.0
    if clip:
        norm = ttt.ttt_grad_norm(g)
        kw = dict(norm=norm, tau=0.25 * float(norm))
        factor = kw["tau"] / float(norm.double())
    ttt.ttt_adamw(w, g, ms, vs, 11, 1e-2, tops=tops, seed=99, **kw, **HYPER)
    vm, vv = ttt.ttt_adamw_values(ms, tops, 1), ttt.ttt_adamw_values(vs, tops, 2)
    for i, s in enumerate(SHAPES):
        n = math.prod(s)
        if n == 0:
            continue
        om = values(before[0][i].reshape(-1), before[2][i][0], 127).astype(np.float64)
        ov = values(before[1][i].reshape(-1), before[2][i][1], 255).astype(np.float64)
        gd = g[i].double().cpu().numpy().reshape(-1) * factor
        m1 = (0.9 * om + (1 - 0.9) * gd).astype(np.float32)
        v1 = (0.999 * ov + (1 - 0.999) * gd * gd).astype(np.float32)
        r = bits_of(99, 11, i, n)
        cm, tm = encode(m1, r & 0xFFFF, 127)
        cv, tv = encode(v1, r >> 16, 255)
        assert np.array_equal(tops[i].cpu().numpy(), np.stack([tm, tv])), i
        assert np.array_equal(ms[i].cpu().numpy().reshape(-1), cm), i
        assert np.array_equal(vs[i].cpu().numpy().reshape(-1), cv), i
        assert np.array_equal(vm[i].cpu().numpy().reshape(-1), values(cm, tm, 127))
        assert np.array_equal(vv[i].cpu().numpy().reshape(-1), values(cv, tv, 255))
        assert vm[i].shape == s and bool((vv[i] >= 0).all())
        # the weights move by the moments before they became codes
        want = step64(ow[i].cpu(), torch.from_numpy(gd).view(s), torch.from_numpy(om).view(s), torch.from_numpy(ov).view(s),
                      11, 1e-2, **HYPER)
        err = 2 * U32 * want[0].abs() + U32 * ow[i].double().cpu().abs() + want[3].abs() * 18 * U32
        assert_close(w[i], want[0], err + half_step(wdt) * (want[0].abs() + err), "w")


def test_codes_hold_16_and_32_octaves_and_keep_the_expectation():
    """One block, moments that the recurrence leaves as they are (betas near 1, gradients equal to the moment's root):
    the mean over seeds of what is held is the value, to 5 standard errors of a step of at most 1/8 of it. (Below the
    smallest value of the block the step is that value.)"""
    n, seeds = 256, 400
    x = torch.exp2(-torch.linspace(0, 17, n)).cuda() * 3.0
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    for s in range(seeds):
        w, m, v = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda"), None
        v = torch.zeros_like(m)
        tops = torch.zeros((2, 1), dtype=torch.int16, device="cuda")
        ttt.ttt_adamw([w], [x], [m], [v], 1, 0.0, betas=(0.0, 0.0), eps=1e-8, weight_decay=0.0, tops=[tops], seed=s)
        held = ttt.ttt_adamw_values([m], [tops], 1)[0]
        total += held.double()
        if s == 0:
            # v = x^2 spans 34 octaves: its smallest values are held as the block's least
            hv = ttt.ttt_adamw_values([v], [tops], 2)[0].double()
            sq = x.double() ** 2
            big = sq > 2.0 ** -31 * sq.max()
            assert bool((hv > 0).all()) and float(((hv - sq).abs() / sq)[big].max()) <= 1 / 8
    mean = total / seeds
    least = 3.0 * 2.0 ** -15.9
    step = torch.maximum(x.double() / 8, torch.tensor(least, device="cuda", dtype=torch.float64))
    assert bool(((mean - x.double()).abs() <= 5 * 0.5 * step / math.sqrt(seeds)).all())


def test_the_random_bits_are_even():
    """Every one of the 32 bits over 2^18 elements, and between the bits of neighbours and of neighbouring seeds, steps
    and tensors: a share within 6 standard deviations (2^-9 / 2) of one half."""
    n = 1 << 18
    base = bits_of(1, 2, 3, n)
    for other in (None, np.roll(base, 1), bits_of(2, 2, 3, n), bits_of(1, 3, 3, n), bits_of(1, 2, 4, n), base >> 16):
        x = base if other is None else base ^ other
        for b in range(32 if other is None or other.max() >= 1 << 16 else 16):
            assert abs(((x >> b) & 1).mean() - 0.5) <= 6 * 0.5 / math.sqrt(n), b


def test_gradients_that_are_not_finite():
    """An element's own moments and weight take the infinity or NaN; elsewhere fp32 moments stay right, and the block of
    8-bit ones it stands in keeps a top that says so."""
    for bad in (float("nan"), float("inf"), -float("inf")):
        n = 1000
        g = torch.full((n,), 1e-3, device="cuda")
        g[300] = bad
        w = torch.ones(n, device="cuda")
        m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        ttt.ttt_adamw([w], [g], [m], [v], 1, 1e-2, norm=ttt.ttt_grad_norm([g]), tau=1.0)
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[300] = False
        assert bool(w[keep].isfinite().all()) and not bool(m[300].isfinite()) and bool(m[keep].isfinite().all())
        assert bool(w[300].isnan())
        w = torch.ones(n, device="cuda")
        m8, v8 = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
        tops = torch.zeros((2, 4), dtype=torch.int16, device="cuda")
        ttt.ttt_adamw([w], [g], [m8], [v8], 1, 1e-2, tops=[tops])
        got = ttt.ttt_adamw_values([m8], [tops], 1)[0]
        assert not bool(got[300].isfinite()) and bool(w[keep].isfinite().all())
        assert math.isnan(bad) == bool(got[300].isnan())
        assert bool(torch.cat([got[:256], got[512:]]).isfinite().all()) and bool((got[:256] > 9e-5).all())


def test_step_and_rate_on_the_device_in_replays():
    for bits in (32, 8):
        gen = torch.Generator().manual_seed(4)
        w0, g = torch.randn(5000, generator=gen).cuda(), torch.randn(5000, generator=gen).cuda()
        kind = torch.float32 if bits == 32 else torch.uint8

        def state():
            return [w0.clone(), torch.zeros(5000, dtype=kind, device="cuda"), torch.zeros(5000, dtype=kind, device="cuda"),
                    torch.zeros((2, 20), dtype=torch.int16, device="cuda")]

        def run(s, step, lr):
            ttt.ttt_adamw([s[0]], [g], [s[1]], [s[2]], step, lr, tops=[s[3]] if bits == 8 else None, seed=3, **HYPER)

        step, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.full((1,), 1e-2, device="cuda")
        a, b = state(), state()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            run(state(), step, lr)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run(a, step, lr)
        for t in range(1, 5):
            rate = 1e-2 / t
            step.fill_(t)
            lr.fill_(rate)
            graph.replay()
            torch.cuda.synchronize()
            run(b, t, float(np.float32(rate)))
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_many_tensors_and_none():
    """More tensors than one launch takes, with empty ones among them: each as it would be alone in its place."""
    gen = torch.Generator().manual_seed(8)
    sizes = [0 if i % 17 == 3 else 1 + i * 13 % 700 for i in range(300)]
    for kind in (torch.float32, torch.uint8):
        w = [torch.randn(n, generator=gen).cuda() for n in sizes]
        g = [torch.randn(n, generator=gen).cuda() for n in sizes]
        m, v = ([torch.zeros(n, dtype=kind, device="cuda") for n in sizes] for _ in range(2))
        tops = [torch.zeros((2, -(-n // 256)), dtype=torch.int16, device="cuda") for n in sizes]
        bits8 = kind == torch.uint8
        one = [[t.clone() for t in ts] for ts in (w, m, v, tops)]
        ttt.ttt_adamw(w, g, m, v, 3, 1e-2, tops=tops if bits8 else None, seed=1, **HYPER)
        for i, n in enumerate(sizes):
            if i % 29 and n:
                continue
            # a list in which the others are empty leaves tensor i its number
            e = [torch.empty(0, device="cuda")] * i
            e8 = [torch.empty(0, dtype=kind, device="cuda")] * i
            et = [torch.empty((2, 0), dtype=torch.int16, device="cuda")] * i
            ttt.ttt_adamw(e + [one[0][i]], e + [g[i]], e8 + [one[1][i]], e8 + [one[2][i]], 3, 1e-2,
                          tops=et + [one[3][i]] if bits8 else None, seed=1, **HYPER)
            for a, b in zip((w, m, v, tops), one):
                assert torch.equal(a[i], b[i]), i
    ttt.ttt_adamw([], [], [], [], 1, 1e-3)
    assert ttt.ttt_adamw_values([], [], 1) == []


def test_elements_past_32_bits():
    """A tensor of 2^31 + 5000 elements: its last chunk and those around the border are what their formula gives."""
    n = (1 << 31) + 5000
    g = torch.Generator(device="cuda").manual_seed(1)
    w, grad = torch.empty(n, dtype=BF16, device="cuda"), torch.empty(n, dtype=BF16, device="cuda")
    for t in (w, grad):
        t[:5000] = torch.randn(5000, generator=g, device="cuda")
        t[5000:(1 << 31) - 5000] = 0.5
        t[(1 << 31) - 5000:] = torch.randn(10000, generator=g, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    tops = torch.zeros((2, -(-n // 256)), dtype=torch.int16, device="cuda")
    at = [slice(0, 4096), slice((1 << 31) - 4096, 1 << 31), slice(1 << 31, n)]
    old = [w[a].clone() for a in at]
    ttt.ttt_adamw([w], [grad], [m], [v], 2, 1e-2, tops=[tops], seed=5, **HYPER)
    for a, ow in zip(at, old):
        gd = grad[a].double().cpu().numpy()
        m1, v1 = ((1 - 0.9) * gd).astype(np.float32), ((1 - 0.999) * gd * gd).astype(np.float32)
        key = mix((5 + GOLDEN * mix(2)) & 0xFFFFFFFF)
        key = mix((key + GOLDEN) & 0xFFFFFFFF)
        e = np.arange(a.start, a.stop, dtype=np.uint64) & np.uint64(0xFFFFFFFF)
        r = mix((np.uint64(key) + e * np.uint64(GOLDEN)) & np.uint64(0xFFFFFFFF)).astype(np.int64)
        cm, tm = encode(m1, r & 0xFFFF, 127)
        cv, tv = encode(v1, r >> 16, 255)
        blocks = slice(a.start // 256, -(-a.stop // 256))
        assert np.array_equal(tops[0, blocks].cpu().numpy(), tm) and np.array_equal(tops[1, blocks].cpu().numpy(), tv)
        assert np.array_equal(m[a].cpu().numpy(), cm) and np.array_equal(v[a].cpu().numpy(), cv)
        want = step64(ow, grad[a], torch.zeros_like(ow), torch.zeros_like(ow), 2, 1e-2, **HYPER)
        err = 2 * U32 * want[0].abs() + U32 * ow.double().abs() + want[3].abs() * 18 * U32
        assert_close(w[a], want[0].cpu(), (err + half_step(BF16) * (want[0].abs() + err)).cpu(), "w")
    vals = ttt.ttt_adamw_values([m], [tops], 1)[0]
    assert np.array_equal(vals[at[2]].cpu().numpy(), values(m[at[2]].cpu().numpy(), tops[0, (1 << 31) // 256:].cpu().numpy(), 127))


def test_refusals_on_the_device():
    x, m = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    v, g = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    c = torch.zeros(10, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="sizes"):
        ttt.ttt_adamw([x], [g[:9]], [m], [v], 1, 1e-3)
    with pytest.raises(ValueError, match="must be torch.float32"):
        ttt.ttt_adamw([x], [g], [m.double()], [v], 1, 1e-3)
    with pytest.raises(ValueError, match="must be torch.uint8"):
        ttt.ttt_adamw([x], [g], [c], [v], 1, 1e-3, tops=[torch.zeros((2, 1), dtype=torch.int16, device="cuda")])
    with pytest.raises(ValueError, match=r"\[2\]\[ceil"):
        ttt.ttt_adamw([x], [g], [c], [c.clone()], 1, 1e-3, tops=[torch.zeros((2, 2), dtype=torch.int16, device="cuda")])
    with pytest.raises(ttt.TTTError, match="overlaps"):
        ttt.ttt_adamw([x], [x], [m], [v], 1, 1e-3)
    with pytest.raises(ttt.TTTError, match="overlaps"):
        ttt.ttt_adamw([x], [g], [m], [m], 1, 1e-3)
    with pytest.raises(ttt.TTTError, match="step"):
        ttt.ttt_adamw([x], [g], [m], [v], 0, 1e-3)
    with pytest.raises(ValueError, match="one element"):
        ttt.ttt_adamw([x], [g], [m], [v], torch.ones(2, dtype=torch.int64, device="cuda"), 1e-3)
    with pytest.raises(ValueError, match="shape"):
        ttt.ttt_adamw([x], [g], [m], [v], 1, 1e-3, norm=torch.ones((), device="cuda"))

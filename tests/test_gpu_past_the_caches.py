"""The variants that large arrays take, which read and write past the caches' keeping from 512 MiB on: the step with fp32
moments, the values of 8-bit moments, and the gradients' elementwise pass, each compared in full with 64 bits."""
import math

import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.block_util import U32, assert_close, half_step
from tests.test_gpu_adamw import HYPER, step64
from tests.test_gpu_linear import act64, d_act64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
PAST = 512 << 20  # bytes


def bounded(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), int(bad.reshape(-1).nonzero()[0]))


def spaced(sizes, dtype, fill, gap=3):
    """Tensors on odd elements of one buffer, which holds 77 between them."""
    buf = torch.full((sum(sizes) + gap * (len(sizes) + 1),), 77.0, dtype=dtype, device="cuda")
    out, at = [], gap
    for n in sizes:
        out.append(buf[at:at + n])
        out[-1].copy_(fill(n))
        at += n + gap
    return buf, out


@pytest.mark.parametrize("wdt,gdt,copied", [(F32, BF16, True), (BF16, F32, False)])
def test_step_with_fp32_moments(wdt, gdt, copied):
    """The bounds of test_moments_in_fp32."""
    sizes = [39_000_000 + 1235, 5000]
    assert sum(sizes) * ((4 if wdt == F32 else 2) + (4 if gdt == F32 else 2) + 8 + 2 * copied) > PAST
    gen = torch.Generator(device="cuda").manual_seed(1)

    def normal(std):
        return lambda n: torch.randn(n, generator=gen, device="cuda").mul_(std)

    (bw, w), (bg, g), (bm, m) = spaced(sizes, wdt, normal(0.5)), spaced(sizes, gdt, normal(1e-2)), spaced(sizes, F32, normal(1e-3))
    bv, v = spaced(sizes, F32, lambda n: normal(1e-2)(n).square_())
    bc, c = spaced(sizes, BF16, lambda n: torch.zeros(n, device="cuda"))
    old = [[t.clone() for t in ts] for ts in (w, m, v)]
    ttt.ttt_adamw(w, g, m, v, 7, 1e-2, copies=c if copied else None, **HYPER)
    for i, n in enumerate(sizes):
        for a in range(0, n, 8_000_000):
            at = slice(a, min(n, a + 8_000_000))
            om, ov, gd = (t[i][at].double() for t in (old[1], old[2], g))
            ww, wm, wv, upd = step64(old[0][i][at], g[i][at], om, ov, 7, 1e-2, **HYPER)
            mags = 0.9 * om.abs() + 0.1 * gd.abs()
            bounded(m[i][at], wm, 4 * U32 * mags, "m")
            bounded(v[i][at], wv, 6 * U32 * (ov + 1e-3 * gd * gd), "v")
            err = 2 * U32 * ww.abs() + U32 * old[0][i][at].double().abs() + upd.abs() * 16 * U32
            err += upd.abs() * 4 * U32 * mags / wm.abs().clamp(min=1e-300)
            bounded(w[i][at], ww, err + half_step(wdt) * (ww.abs() + err), "w")
            if copied:
                bounded(c[i][at], ww, err + half_step(BF16) * (ww.abs() + err), "copy")
    for buf, views in ((bw, w), (bg, g), (bm, m), (bv, v), (bc, c)):
        ends = [0] + [e for t in views for e in (t.storage_offset(), t.storage_offset() + t.numel())] + [buf.numel()]
        assert all(bool((buf[a:b] == 77.0).all()) for a, b in zip(ends[::2], ends[1::2])), "written between the tensors"


@pytest.mark.parametrize("moment", [1, 2])
def test_values_of_8_bit_moments(moment):
    """Every code under tops of the whole range, from where all its values are 0 to where the highest are NaN."""
    sizes = [113_000_000 + 77, 300]
    assert sum(sizes) * 5 > PAST
    gen = torch.Generator(device="cuda").manual_seed(2)
    most = 127 if moment == 1 else 255
    codes = [torch.randint(0, 256, (n,), generator=gen, device="cuda", dtype=torch.uint8) for n in sizes]
    tops = [torch.randint(0, 0x7FD, (2, -(-n // 256)), generator=gen, device="cuda", dtype=torch.int16) for n in sizes]
    _, out = spaced(sizes, F32, lambda n: torch.zeros(n, device="cuda"))
    ttt.ttt_adamw_values(codes, tops, moment, out=out)
    for c, t, o in zip(codes, tops, out):
        for a in range(0, c.numel(), 1 << 25):
            part = c[a:a + (1 << 25)].int()
            top = t[moment - 1, a // 256:].int().repeat_interleave(256)[:part.numel()]
            k = part & most
            bits = torch.where(k > 0, (top - most + k).clamp(min=0) << 20, 0)
            if moment == 1:
                bits = bits | (part >> 7 << 31)
            assert torch.equal(o[a:a + (1 << 25)].view(torch.int32), bits)


def rows_of(n, bytes_each):
    """Rows of n that together just pass the border, not a whole number of a workgroup's."""
    return PAST // (n * bytes_each) + 14


def products(q, e, x, w, dt, dx, dw, what):
    """As check_products of test_gpu_linear.py, on the device."""
    M = x.shape[0]
    want = sum(a @ b.double() for a, b in zip(q, w))
    n = sum(a.shape[1] for a in q)
    err = sum((b + 2 * (n + 3) * U32 * (a.abs() + b)) @ c.double().abs() for a, b, c in zip(q, e, w)) + 2 * U32 * want.abs()
    assert_close(dx, want.cpu(), (err + half_step(dt) * (want.abs() + err)).cpu(), what + " dx")
    for a, b, got in zip(q, e, dw):
        want = a.T @ x.double()
        err = (b + 2 * (M + 3) * U32 * (a.abs() + b)).T @ x.double().abs() + 2 * U32 * want.abs()
        assert_close(got, want.cpu(), (err + half_step(dt) * (want.abs() + err)).cpu(), what + " dw")


def column_sums(q, e, got, what):
    M = q.shape[0]
    want = q.sum(0)
    err = (e + 2 * (M + 3) * U32 * (q.abs() + e)).sum(0) + 2 * U32 * want.abs()
    assert_close(got, want.cpu(), err.cpu(), what)


@pytest.mark.parametrize("N", [8192, 5003])
@pytest.mark.parametrize("dt,ydt,act", [(BF16, BF16, "gelu"), (BF16, F32, "silu"), (BF16, F32, None), (F32, F32, "silu")])
def test_pass_of_linear_gradients(dt, ydt, act, N):
    """Without the bias' sums (end to end where the width is whole pieces), and with them (by rows): the same bits, and
    those the formula's."""
    K = 24
    M = rows_of(N, (4 if ydt == F32 else 2) + (2 if act else 1) * (4 if dt == F32 else 2))
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, w = torch.randn((M, K), generator=gen, device="cuda").to(dt), torch.randn((N, K), generator=gen, device="cuda").to(dt)
    dy = torch.randn((M, N), generator=gen, device="cuda").to(ydt)
    pre = torch.randn((M, N), generator=gen, device="cuda").mul_(2).to(dt) if act else None
    got = ttt.ttt_linear_grad(dy, x, w, act=act, pre=pre, bias=True)
    alone = ttt.ttt_linear_grad(dy, x, w, act=act, pre=pre)
    assert torch.equal(got.dx, alone.dx) and torch.equal(got.dw, alone.dw)
    q = dy.double() * (d_act64(pre.double(), act) if act else 1.0)
    e = 64 * U32 * dy.double().abs() + 2 * U32 * q.abs() if act else torch.zeros_like(q)
    made = act or ydt != dt
    er = e + half_step(dt) * (q.abs() + e) if made else e
    products([q], [er + 2 * U32 * q.abs()], x, [w], dt, got.dx, [got.dw], str((dt, ydt, act)))
    column_sums(q, e + 2 * U32 * q.abs(), got.dbias, "dbias")


@pytest.mark.parametrize("f", [8192, 5003])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_pass_of_gated_gradients(dt, f):
    K = 24
    M = rows_of(f, 5 * (4 if dt == F32 else 2))
    gen = torch.Generator(device="cuda").manual_seed(4)

    def normal(shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dt)

    x, wg, wu = normal((M, K)), normal((f, K)), normal((f, K))
    dz, g, u = normal((M, f)), normal((M, f), 2.0), normal((M, f))
    got = ttt.ttt_gated_grad(dz, x, wg, wu, g, u, bias=True)
    alone = ttt.ttt_gated_grad(dz, x, wg, wu, g, u)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], alone[:3]))
    zd, ud, gd = dz.double(), u.double(), g.double()
    q = [zd * ud * d_act64(gd, "silu"), zd * act64(gd, "silu")]
    e = [64 * U32 * (zd * ud).abs() + 3 * U32 * q[0].abs(), 16 * U32 * (zd * gd).abs() + 2 * U32 * q[1].abs()]
    er = [b + half_step(dt) * (a.abs() + b) for a, b in zip(q, e)]
    products(q, er, x, [wg, wu], dt, got.dx, [got.dw_gate, got.dw_up], str(dt))
    column_sums(q[0], e[0], got.db_gate, "db_gate")
    column_sums(q[1], e[1], got.db_up, "db_up")
    assert math.isfinite(float(got.dx.float().norm()))

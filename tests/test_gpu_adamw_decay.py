"""The decay of fp32 moments: their weights and those of the gradient add up to one, also where a beta is not near an
fp32 number."""
import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.block_util import U32, assert_close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BETAS = [(0.9, 0.9999), (0.99, 0.99999), (0.8, 0.999999), (0.3, 0.0), (0.0, 0.1), (0.95, 1 - 1e-8)]


@pytest.mark.parametrize("betas", BETAS)
def test_without_a_gradient_the_moments_are_the_decayed_ones_rounded_once(betas):
    """g = 0: m' = beta1 m and v' = beta2 v, one rounding of the exact products. (A beta rounded to fp32 first is off by
    up to U / 2 more, of values that keep it step after step.)"""
    g = torch.Generator().manual_seed(1)
    n = 20000
    m = torch.randn(n, generator=g).cuda()
    v = torch.rand(n, generator=g).cuda() + 1e-3
    w, zero = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    wm, wv = betas[0] * m.double(), betas[1] * v.double()
    ttt.ttt_adamw([w], [zero], [m], [v], 5, 0.0, betas=betas)
    once = U32 * (1 + 2.0 ** -16)
    assert_close(m, wm.cpu(), once * wm.abs().cpu(), "m")
    assert_close(v, wv.cpu(), once * wv.abs().cpu(), "v")


def test_infinite_moments_stay_infinite():
    """As the products of the definition: beta times infinity, plus what is finite."""
    for betas in BETAS[:3] + BETAS[5:]:
        m = torch.tensor([float("inf"), -float("inf"), float("nan"), 1.0], device="cuda")
        v = torch.tensor([float("inf"), float("inf"), float("nan"), 1.0], device="cuda")
        w, g = torch.ones(4, device="cuda"), torch.full((4,), 0.5, device="cuda")
        ttt.ttt_adamw([w], [g], [m], [v], 2, 1e-3, betas=betas)
        assert m.tolist()[:2] == [float("inf"), -float("inf")] and v.tolist()[:2] == [float("inf")] * 2
        assert bool(m[2].isnan()) and bool(v[2].isnan()) and bool(torch.stack([m[3], v[3], w[3]]).isfinite().all())


def test_the_factors_with_every_type():
    for wdt, gdt in ((F32, BF16), (BF16, BF16), (BF16, F32)):
        g = torch.Generator().manual_seed(4)
        n = 5000
        w, d = torch.randn(n, generator=g).to(wdt).cuda(), torch.randn(n, generator=g).to(gdt).cuda()
        m, v = torch.randn(n, generator=g).cuda(), torch.rand(n, generator=g).cuda()
        om, ov = m.double(), v.double()
        ttt.ttt_adamw([w], [d], [m], [v], 4, 1e-3, betas=(0.8, 0.9999))
        x = d.double()
        wm, wv = 0.8 * om + 0.2 * x, 0.9999 * ov + (1 - 0.9999) * x * x
        # decayed: two roundings; the gradient's term: its factor, products, and the sum
        assert_close(m, wm.cpu(), (U32 * (2.01 * 0.8 * om.abs() + 3 * 0.2 * x.abs())).cpu(), "m")
        assert_close(v, wv.cpu(), (U32 * (2.01 * ov + 4 * 1e-4 * x * x)).cpu(), "v")

"""The AdamW step where the root of the second moment or eps leaves fp32's normal numbers, which the hardware's root and
reciprocal take as zero: the formula in 64 bits, with the moments as they are held (fp32)."""
import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.block_util import U32, assert_close

pytestmark = pytest.mark.gpu

F32 = torch.float32


def moved64(w, m, v, step, lr, betas, eps, decay):
    """The weight from the new moments."""
    b1, b2 = betas
    upd = lr * (m.double() / (1 - b1 ** step)) / (torch.sqrt(v.double() / (1 - b2 ** step)) + eps)
    return w.double() * (1 - lr * decay) - upd, upd


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [2.0 ** -127, 1e-42, 2.0 ** -149, 1e-60, 5e-324])
def test_elements_that_never_had_a_gradient(eps, bits):
    """Both moments zero: the step is 0 / (0 + eps) = 0 for every eps above 0, and the weight only shrinks (one rounding
    of the factor, one of the result)."""
    n = 5000
    w = torch.randn(n, generator=torch.Generator().manual_seed(1)).cuda()
    kind = F32 if bits == 32 else torch.uint8
    m, v = (torch.zeros(n, dtype=kind, device="cuda") for _ in range(2))
    tops = [torch.zeros((2, -(-n // 256)), dtype=torch.int16, device="cuda")] if bits == 8 else None
    want = w.double() * (1 - 1e-2 * 0.1)
    ttt.ttt_adamw([w], [torch.zeros(n, device="cuda")], [m], [v], 3, 1e-2, eps=eps, weight_decay=0.1, tops=tops)
    assert_close(w, want.cpu(), 2 * U32 * want.abs().cpu(), "w")
    assert not m.any() and not v.any()


@pytest.mark.parametrize("eps", [2.0 ** -126, 2.0 ** -130, 2.0 ** -140, 2.0 ** -100, 2.0 ** -90])
def test_eps_alone_below_the_step(eps):
    """A second moment of zero and a first one that is not: lr m / eps, at denominators on both sides of where they are
    scaled. The moments' decay is 1/2 and their bias 3/4, which fp32 holds; the rate, the quotient's factors and the
    reciprocal (1 ulp, two half steps) are some roundings off, 16 together, as in the other tests of the step."""
    w = torch.linspace(-1, 1, 3001).cuda()
    m = (torch.randn(3001, generator=torch.Generator().manual_seed(2)) * 2.0 ** 8 * eps).cuda()
    v, old = torch.zeros_like(m), m.clone()
    want, upd = moved64(w, 0.5 * old, v, 2, 1e-3, (0.5, 0.5), eps, 0.0)
    # a decayed moment may itself be below the normal numbers
    lost = 1e-3 * 2.0 ** -149 / 0.75 / eps
    ttt.ttt_adamw([w], [torch.zeros_like(w)], [m], [v], 2, 1e-3, betas=(0.5, 0.5), eps=eps, weight_decay=0.0)
    assert_close(w, want.cpu(), (16 * U32 * upd.abs() + U32 * want.abs() + lost).cpu(), "w")


@pytest.mark.parametrize("eps", [0.0, 1e-12, 1e-10, 1e-8])
@pytest.mark.parametrize("b2", [0.5, 0.999, 0.99999999])
def test_second_moments_below_the_normal_numbers(b2, eps):
    """v held as a denormal, whose root over (1 - b2)^1/2 may count beside eps."""
    n = 2000
    v = torch.full((n,), 2.0 ** -130, device="cuda") * torch.arange(1, n + 1, device="cuda").float() / 64
    m = torch.full((n,), 1e-14, device="cuda")
    w = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    ttt.ttt_adamw([w], [g], [m], [v], 1, 1e-3, betas=(0.5, b2), eps=eps, weight_decay=0.0)
    want, upd = moved64(torch.zeros_like(w), m, v, 1, 1e-3, (0.5, b2), eps, 0.0)
    assert bool((v < 2.0 ** -120).all())
    assert_close(w, want.cpu(), 16 * U32 * upd.abs().cpu(), "w")

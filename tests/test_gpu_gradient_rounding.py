"""What the bf16 gradients round: q, dg and du once to the products' type, and each result once, nothing between. With
ReLU and no scale q, dg and du are exact before that rounding (signs, and products of two bf16 numbers), so the rounded
ones are known to the bit and the products' own error is all that is left beside a result's rounding."""
import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.block_util import U32, assert_close, half_step

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def close(got, pairs, what):
    """got: the sum of a @ b over pairs, one rounding to bf16 and 2 (n + 3) of fp32 in the sums."""
    want = sum(a.double() @ b.double() for a, b in pairs)
    n = sum(a.shape[1] for a, _ in pairs)
    err = 2 * (n + 3) * U32 * sum(a.double().abs() @ b.double().abs() for a, b in pairs) + U32 * want.abs()
    assert_close(got, want.cpu(), (err + half_step(BF16) * (want.abs() + err)).cpu(), what)
    return float((got.double() - want).norm() / want.norm())


# tiles of 64, of 128, of 256, and odd rows
SIZES = [(300, 200, 136), (4125, 72, 2480), (14479, 520, 160), (700, 513, 1027)]


def normal(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("ydt,act", [(F32, None), (F32, "relu"), (BF16, "relu")])
def test_linear(M, K, N, ydt, act):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x, w, dy, pre = normal(g, M, K), normal(g, N, K), normal(g, M, N, dtype=ydt), normal(g, M, N)
    got = ttt.ttt_linear_grad(dy, x, w, act=act, pre=pre if act else None)
    q = (dy * (pre > 0) if act else dy).to(BF16)
    errors = close(got.dx, [(q, w)], "dx"), close(got.dw, [(q.T, x)], "dw")
    # a bf16 rounding is at most 2^-8 of a number, at random some 0.43 of that in the mean square
    assert max(errors) <= 0.6 * half_step(BF16)


@pytest.mark.parametrize("M,K,f", SIZES)
def test_gated(M, K, f):
    gen = torch.Generator(device="cuda").manual_seed(M + f)
    x, wg, wu, dz, g, u = normal(gen, M, K), normal(gen, f, K), normal(gen, f, K), *(normal(gen, M, f) for _ in range(3))
    got = ttt.ttt_gated_grad(dz, x, wg, wu, g, u, act="relu")
    dg = (dz.float() * u.float() * (g > 0)).to(BF16)
    du = (dz.float() * g.float().clamp(min=0)).to(BF16)
    errors = (close(got.dx, [(dg, wg), (du, wu)], "dx"), close(got.dw_gate, [(dg.T, x)], "dw_gate"),
              close(got.dw_up, [(du.T, x)], "dw_up"))
    assert max(errors) <= 0.6 * half_step(BF16)


def test_fp32_operands_round_nothing_to_fewer_bits():
    """The form for a caller who wants the fp32 gradient of an fp32 stream as it is: everything in fp32."""
    g = torch.Generator(device="cuda").manual_seed(5)
    M, K, N = 1000, 264, 520
    x, w, dy = normal(g, M, K), normal(g, N, K), normal(g, M, N, dtype=F32)
    got = ttt.ttt_linear_grad(dy, x.float(), w.float())
    want = dy.double() @ w.double()
    err = 2 * (N + 3) * U32 * (dy.double().abs() @ w.double().abs()) + 2 * U32 * want.abs()
    assert_close(got.dx, want.cpu(), err.cpu(), "dx")

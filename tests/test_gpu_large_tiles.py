"""The products' kernels by the variant that runs them: each tile, with k whole and split, of each product and type, over
several slabs of k and with ragged last tiles. A case first asks which variant its sizes take, so that a change of the
rule cannot leave one untested; then it is compared with the formulas in 64 bits, element by element, with the bounds of
test_gpu_linear.py.

The sizes are about the smallest that the rule sends there. DIRECT ones have whole 16-byte rows, COPIED ones are odd and
copied first, GENERAL ones odd and not copied."""
import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.test_gpu_linear import gated_case, gated_grad_case, linear_case, linear_grad_case, make

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
WHOLE, SPLIT = False, True

# product, type, tile, k split, (rows, in, out)
DIRECT = [
    ("linear", BF16, 64, SPLIT, (132, 2240, 48)), ("linear", BF16, 128, WHOLE, (16850, 344, 136)),
    ("linear", BF16, 128, SPLIT, (4183, 4456, 80)), ("linear", BF16, 256, WHOLE, (13276, 336, 528)),
    ("linear", BF16, 256, SPLIT, (10923, 5288, 136)),
    ("linear", F32, 64, SPLIT, (105, 456, 40)), ("linear", F32, 128, WHOLE, (8073, 160, 904)),
    ("linear", F32, 128, SPLIT, (8641, 2144, 72)),
    ("gated", BF16, 64, SPLIT, (132, 2240, 48)), ("gated", BF16, 128, WHOLE, (16550, 328, 72)),
    ("gated", BF16, 128, SPLIT, (4118, 5104, 40)), ("gated", BF16, 256, WHOLE, (572, 328, 6688)),
    ("gated", BF16, 256, SPLIT, (129, 7440, 4496)),
    ("gated", F32, 64, SPLIT, (105, 456, 40)), ("gated", F32, 128, WHOLE, (471, 160, 7736)),
    ("gated", F32, 128, SPLIT, (8487, 2392, 40)),
    ("linear_dx", BF16, 64, SPLIT, (235, 40, 1920)), ("linear_dx", BF16, 128, WHOLE, (17185, 144, 320)),
    ("linear_dx", BF16, 128, SPLIT, (4167, 72, 4944)), ("linear_dx", BF16, 256, WHOLE, (16682, 392, 368)),
    ("linear_dx", BF16, 256, SPLIT, (131, 8840, 7696)),
    ("linear_dx", F32, 64, SPLIT, (113, 40, 456)), ("linear_dx", F32, 128, WHOLE, (3586, 2096, 160)),
    ("linear_dx", F32, 128, SPLIT, (9145, 72, 2160)),
    ("linear_dw", BF16, 64, SPLIT, (1600, 88, 80)), ("linear_dw", BF16, 128, WHOLE, (332, 8368, 328)),
    ("linear_dw", BF16, 128, SPLIT, (6397, 72, 3272)), ("linear_dw", BF16, 256, WHOLE, (324, 1968, 4200)),
    ("linear_dw", BF16, 256, SPLIT, (14195, 4264, 144)),
    ("linear_dw", F32, 64, SPLIT, (521, 40, 40)), ("linear_dw", F32, 128, WHOLE, (165, 2984, 2440)),
    ("linear_dw", F32, 128, SPLIT, (2361, 72, 8248)),
    ("gated_dx", BF16, 64, SPLIT, (103, 56, 960)), ("gated_dx", BF16, 128, WHOLE, (16745, 144, 184)),
    ("gated_dx", BF16, 128, SPLIT, (4125, 72, 2480)), ("gated_dx", BF16, 256, WHOLE, (14479, 520, 160)),
    ("gated_dx", BF16, 256, SPLIT, (4605, 136, 6920)),
    ("gated_dx", F32, 64, SPLIT, (102, 40, 208)), ("gated_dx", F32, 128, WHOLE, (19727, 336, 80)),
    ("gated_dx", F32, 128, SPLIT, (8315, 72, 1208)),
    ("gated_dw", BF16, 64, SPLIT, (1600, 88, 80)), ("gated_dw", BF16, 128, WHOLE, (337, 200, 6624)),
    ("gated_dw", BF16, 128, SPLIT, (7040, 72, 1736)), ("gated_dw", BF16, 256, WHOLE, (336, 5648, 712)),
    ("gated_dw", BF16, 256, SPLIT, (5328, 5768, 144)),
    ("gated_dw", F32, 64, SPLIT, (521, 40, 40)), ("gated_dw", F32, 128, WHOLE, (169, 472, 7224)),
    ("gated_dw", F32, 128, SPLIT, (2119, 4104, 104)),
]
COPIED = [
    ("linear", BF16, 128, WHOLE, (969, 322, 3120)), ("linear", BF16, 256, WHOLE, (3203, 339, 2528)),
    ("linear", BF16, 256, SPLIT, (12365, 5011, 146)), ("linear", F32, 128, WHOLE, (2460, 197, 7969)),
    ("gated", BF16, 128, SPLIT, (2049, 2796, 228)), ("gated", BF16, 256, WHOLE, (6821, 355, 616)),
    ("linear_dx", BF16, 128, SPLIT, (5742, 65, 4292)), ("linear_dx", BF16, 256, WHOLE, (18956, 404, 1263)),
    ("linear_dw", BF16, 128, WHOLE, (326, 6273, 449)), ("linear_dw", BF16, 256, SPLIT, (8327, 8217, 139)),
    ("linear_dw", F32, 128, WHOLE, (214, 2398, 4877)),
    ("gated_dx", BF16, 256, SPLIT, (11798, 138, 2734)), ("gated_dx", F32, 128, WHOLE, (14364, 453, 130)),
    ("gated_dw", BF16, 256, WHOLE, (1266, 849, 4712)), ("gated_dw", F32, 128, SPLIT, (3338, 69, 4316)),
]
GENERAL = [
    ("linear", BF16, 128, WHOLE, (18023, 527, 85)), ("linear", BF16, 128, SPLIT, (6260, 1610, 69)),
    ("linear", F32, 128, WHOLE, (2822, 161, 2517)), ("linear", F32, 128, SPLIT, (8561, 2049, 65)),
    ("gated", BF16, 128, SPLIT, (3405, 2890, 44)), ("gated", F32, 128, WHOLE, (13002, 161, 269)),
    ("linear_dx", BF16, 128, SPLIT, (116, 1908, 8000)), ("linear_dx", F32, 128, WHOLE, (906, 7674, 162)),
    ("linear_dw", BF16, 128, SPLIT, (5942, 3477, 68)), ("linear_dw", F32, 128, SPLIT, (2836, 7115, 68)),
    ("gated_dx", BF16, 128, SPLIT, (102, 7323, 1151)), ("gated_dx", F32, 128, WHOLE, (1564, 4613, 80)),
    ("gated_dw", BF16, 128, SPLIT, (8561, 2049, 65)), ("gated_dw", F32, 128, WHOLE, (161, 477, 7482)),
]
CASES = [("direct", False, *c) for c in DIRECT] + [("direct", True, *c) for c in COPIED] + [("general", False, *c) for c in GENERAL]


def name(c):
    return f"{c[0]}{'-copied' * c[1]}-{c[2]}-{str(c[3])[6:]}-{c[4]}{'-split' * c[5]}"


def k_of(product, M, K, N):
    return M if product.endswith("dw") else {"linear_dx": N, "gated_dx": 2 * N}.get(product, K)


@pytest.mark.parametrize("kernel,copied,product,dt,tile,split,size", CASES, ids=map(name, CASES))
def test_variant(kernel, copied, product, dt, tile, split, size):
    plan = ttt.ttt_dense_plan(product, *size, dt, q_made=True)
    assert (plan["kernel"], plan["copies"] > 0, plan["tile"], plan["splits"] > 1) == (kernel, copied, tile, split), plan
    slab = 64 if dt == BF16 else 32
    assert k_of(product, *size) / slab / plan["splits"] > 4, "more slabs than a ring holds"
    if product == "linear":
        linear_case(*size, dt, F32, "gelu", True, True, 0.5, 0)
        linear_case(*size, dt, dt, None, False, True, 1.0, 0)
    elif product == "gated":
        gated_case(*size, dt, "silu", True, 0)
    elif product.startswith("linear"):
        linear_grad_case(*size, dt, F32, "silu", 0.5, 0, accumulate=True)
    else:
        gated_grad_case(*size, dt, "gelu", 0, accumulate=True)


def test_the_variants_are_all_there():
    """Every tile of every product and type, whole and split, straight to LDS."""
    want = {(p, dt, t, s) for p in ("linear", "gated", "linear_dx", "linear_dw", "gated_dx", "gated_dw")
            for dt, tiles in ((BF16, (64, 128, 256)), (F32, (64, 128))) for t in tiles for s in (WHOLE, SPLIT)}
    # tiles of 64 with k whole are those of most sizes of test_gpu_linear.py
    assert want - {c[:4] for c in DIRECT} == {c for c in want if c[2] == 64 and c[3] == WHOLE}


@pytest.mark.parametrize("M,K,N,split", [(13276, 336, 528, False), (10923, 5288, 136, True)])
def test_in_place_residual_in_tiles_of_256(M, K, N, split):
    plan = ttt.ttt_dense_plan("linear", M, K, N, BF16)
    assert plan["tile"] == 256 and (plan["splits"] > 1) == split
    g = torch.Generator().manual_seed(1)
    x, w = make((M, K), BF16, g).cuda(), make((N, K), BF16, g, 1 / 16).cuda()
    for dt in (F32, BF16):
        h = make((M, N), dt, g).cuda()
        want = ttt.ttt_linear(x, w, residual=h)
        assert torch.equal(ttt.ttt_linear(x, w, residual=h, y=h), want)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_the_same_bits_again_in_large_tiles(dt):
    """Each product in its largest tile, split, and whole: two calls, and one among others on another stream."""
    g = torch.Generator().manual_seed(2)
    side = torch.cuda.Stream()
    for M, K, N in [(14195, 4264, 144), (4605, 136, 6920)] if dt == BF16 else [(8641, 2144, 72), (2119, 4104, 104)]:
        x, w, wu = make((M, K), dt, g).cuda(), make((N, K), dt, g, 0.02).cuda(), make((N, K), dt, g, 0.02).cuda()
        dy, pre = make((M, N), dt, g).cuda(), make((M, N), dt, g).cuda()

        def all_of_them(stream=None):
            return [ttt.ttt_linear(x, w, residual=dy, stream=stream), *ttt.ttt_gated(x, w, wu, keep=True, stream=stream),
                    *ttt.ttt_linear_grad(dy, x, w, act="silu", pre=pre, bias=True, stream=stream),
                    *ttt.ttt_gated_grad(dy, x, w, wu, pre, dy, bias=True, stream=stream)]

        want = all_of_them()
        side.wait_stream(torch.cuda.current_stream())
        other = all_of_them(side)
        again = all_of_them()
        torch.cuda.synchronize()
        for a, b, c in zip(want, other, again):
            assert torch.equal(a, b) and torch.equal(a, c)

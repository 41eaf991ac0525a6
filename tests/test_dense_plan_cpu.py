"""The host-only query of how the plain layers' products run."""
import ctypes

import pytest
import torch

import chunk_wise_weight_amd as ttt

F32, BF16 = torch.float32, torch.bfloat16
PRODUCTS = ("linear", "gated", "linear_dx", "linear_dw", "gated_dx", "gated_dw")


def test_refusals():
    L, n = ttt.lib(), ctypes.c_int()
    q = L.ttt_dense_plan
    assert q(6, 100, 64, 64, 1, 0, n, n, n, n) == -7 and q(-1, 100, 64, 64, 1, 0, n, n, n, n) == -7
    assert q(0, 100, 64, 64, 2, 0, n, n, n, n) == -3
    assert q(0, -1, 64, 64, 1, 0, n, n, n, n) == q(0, 100, 0, 64, 1, 0, n, n, n, n) == -2
    assert q(0, 100, 64, 64, 1, 0, None, None, None, None) == 0
    with pytest.raises(ValueError, match="product must be"):
        ttt.ttt_dense_plan("dx", 1, 1, 1, F32)
    with pytest.raises(ValueError, match="dtype must be"):
        ttt.ttt_dense_plan("linear", 1, 1, 1, torch.float16)
    with pytest.raises(ValueError, match="below 2"):
        ttt.ttt_dense_plan("linear", 1, 1, 1 << 32, F32)


def test_few_rows_and_odd_rows():
    assert ttt.ttt_dense_plan("linear", 1, 9728, 2560, BF16) == {"kernel": "few", "tile": 0, "splits": 1, "copies": 0}
    assert ttt.ttt_dense_plan("gated", 8, 2560, 9728, BF16)["kernel"] == "few"
    assert ttt.ttt_dense_plan("linear", 4099, 1021, 2047, BF16)["copies"] == 2
    # rows of q that is made need no copy
    assert ttt.ttt_dense_plan("linear_dw", 8192, 2560, 9721, BF16, q_made=False)["copies"] == 1
    assert ttt.ttt_dense_plan("linear_dw", 8192, 2560, 9721, BF16, q_made=True)["copies"] == 0
    assert ttt.ttt_dense_plan("linear_dx", 0, 8, 8, F32)["splits"] == 1


@pytest.mark.parametrize("dt", [F32, BF16])
def test_workspaces_hold_the_split_sums(dt):
    """A forward product of whole rows needs at least its tiles' fp32 sums, splits times."""
    n = ctypes.c_size_t()
    for M, K, N in [(132, 2240, 48), (4183, 4456, 80), (10923, 5288, 136), (105, 456, 40), (8641, 2144, 72)]:
        p = ttt.ttt_dense_plan("linear", M, K, N, dt)
        assert ttt.lib().ttt_linear_ws_bytes(M, K, N, 0 if dt == F32 else 1, ctypes.byref(n)) == 0
        tiles = -(-M // p["tile"]) * -(-N // p["tile"])
        assert p["splits"] == 1 or n.value >= tiles * p["splits"] * p["tile"] ** 2 * 4


@pytest.mark.parametrize("product", PRODUCTS)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_launches_stay_within_their_threads(product, dt):
    """A launch of tiles straight to LDS counts its threads in 32 bits, whatever the sizes."""
    widths = [8, 64, 128, 520, 4096, 65536, 1 << 20]
    for M in [17, 256, 5000, 1 << 20, 1 << 25, (1 << 29) + 8, (1 << 31) - 8]:
        for K in widths:
            for N in widths:
                p = ttt.ttt_dense_plan(product, M, K, N, dt, q_made=True)
                if p["kernel"] != "direct":
                    continue
                i, j = {"linear": (N, M), "gated": (2 * N, M), "linear_dw": (K, N), "gated_dw": (K, 2 * N)}.get(product, (K, M))
                tiles = -(-i // p["tile"]) * -(-j // p["tile"])
                assert tiles * p["splits"] * (512 if p["tile"] == 256 else 256) < 1 << 32, (M, K, N, p)

"""Where the plain layers' arrays lie does not matter: operands on any 16 bytes, results, biases, residuals and kept sums
on any element give the bits of a call on fresh tensors, with NaN around every array; and so does a captured call."""
import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.test_gpu_linear import Held, empty, make

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16

# one token, few rows, tiles of 64, 128 and 256 with k whole and split, odd rows that are copied
SIZES = [(1, 512, 264), (13, 264, 520), (300, 520, 392), (4183, 4456, 80), (572, 328, 6688), (10923, 1288, 136), (1500, 1021, 1031)]


def both(x, w, wu, b, r, dy, pre, at, out_at):
    """Every entry point on copies `at` elements into their buffers, results `out_at` elements into theirs."""
    M, N = dy.shape
    K = x.shape[1]
    dt = x.dtype
    held = []

    def place(t, off):
        held.append(Held(t, off))
        return held[-1].t

    def out(shape, dtype=dt):
        held.append(empty(shape, dtype, out_at))
        return held[-1].t

    x, w, wu, dy, pre = (place(t, at) for t in (x, w, wu, dy, pre))
    b, r = place(b, out_at), place(r, out_at)
    y, z, dx, dw, db = out((M, N), r.dtype), out((M, N)), out((M, K)), out((N, K)), out((N,), F32)
    gx, gg, gu = out((M, K)), out((N, K)), out((N, K))
    got = [*ttt.ttt_linear(x, w, b, act="gelu", residual=r, keep=True, y=y), *ttt.ttt_gated(x, w, wu, b, b, keep=True, z=z),
           *ttt.ttt_linear_grad(dy, x, w, act="silu", pre=pre, bias=True, dx=dx, dw=dw, dbias=db),
           *ttt.ttt_gated_grad(dy, x, w, wu, pre, pre, dx=gx, dw_gate=gg, dw_up=gu)[:3]]
    for h in held:
        h.check()
    return [t.clone() for t in got]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_placement(M, K, N, dt):
    g = torch.Generator().manual_seed(M + K + N)
    t = [make(s, d, g, k) for s, d, k in (((M, K), dt, 1.0), ((N, K), dt, K ** -0.5), ((N, K), dt, K ** -0.5), ((N,), dt, 0.3),
                                          ((M, N), F32, 1.0), ((M, N), dt, 1.0), ((M, N), dt, 1.0))]
    want = both(*t, 0, 0)
    assert all(bool(a.isfinite().all()) for a in want)
    piece = 16 // t[0].element_size()
    for at, out_at in ((piece, 0), (3 * piece, 1), (0, 3)):
        for i, (a, b) in enumerate(zip(both(*t, at, out_at), want)):
            assert torch.equal(a, b), (at, out_at, i)


@pytest.mark.parametrize("M,K,N", [(10923, 1288, 136), (5328, 5768, 144), (572, 328, 6688), (1500, 1021, 1031)])
def test_captured_calls_in_large_tiles(M, K, N):
    """Split sums, copies and q in a graph's own memory: every replay is the eager call on what the inputs then hold, also
    with other work and another graph of the same calls between the replays."""
    g = torch.Generator().manual_seed(M)
    x, w, wu = make((M, K), BF16, g).cuda(), make((N, K), BF16, g, 0.02).cuda(), make((N, K), BF16, g, 0.02).cuda()
    dy, pre = make((M, N), F32, g).cuda(), make((M, N), BF16, g).cuda()
    dz = dy.bfloat16()

    def calls():
        return [ttt.ttt_linear(x, w, residual=dy), *ttt.ttt_gated(x, w, wu, keep=True),
                *ttt.ttt_linear_grad(dy, x, w, act="gelu", pre=pre, bias=True), *ttt.ttt_gated_grad(dz, x, w, wu, pre, dz, bias=True)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    got = []
    for graph in graphs:
        with torch.cuda.graph(graph, stream=side):
            got.append(calls())
    for _ in range(3):
        x.mul_(0.5)
        want = calls()
        torch.cuda.synchronize()
        for graph, outs in zip(graphs, got):
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b)

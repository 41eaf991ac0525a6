"""Token embedding and its gradient against the formulas in 64 bits.

Bounds. The lookup is one product in fp32 and one rounding: u + half a step of
the type. The gradient of a table row sums its c tokens in fp32, the longest
way through a piece of 32, then a run of an eighth of the pieces, then eight
sums: at most 31 + ceil(c / 32 / 8) + 1 + 8 additions, then the scale and, when
accumulating, one more addition.
"""
import pytest
import torch

import chunk_wise_weight_amd as ttt
from tests.block_util import U32, Guarded, assert_close, guarded, half_step

F, B16 = torch.float32, torch.bfloat16
gpu = pytest.mark.gpu


def make_ids(B, T, vocab, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "same":
        ids = torch.full((B, T + 1), vocab // 2)
    elif kind == "skewed":
        ids = (torch.exp(torch.rand((B, T + 1), generator=g, dtype=torch.float64) *
                         torch.log(torch.tensor(float(vocab)))) - 1).long().clamp(0, vocab - 1)
    else:
        ids = torch.randint(0, vocab, (B, T + 1), generator=g)
    ids = ids.int()
    if kind == "holes":  # ids outside the table, at the ends of the type too
        bad = torch.rand((B, T + 1), generator=g) < 0.5
        ids[bad] = torch.tensor([-1, vocab, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)[
            torch.randint(0, 4, (int(bad.sum()),), generator=g)]
    return ids[:, :T]


CASES = [  # B, T, vocab, d, kind
    (1, 1, 1, 8, "uniform"), (3, 5, 7, 9, "holes"), (2, 64, 513, 64, "same"), (1, 65, 100, 72, "same"),
    (2, 1000, 50, 100, "skewed"), (3, 411, 512, 1024, "skewed"), (1, 4000, 3, 257, "uniform"),
    (4, 1025, 70001, 40, "skewed"), (1, 2049, 151936, 8, "uniform"), (5, 300, 1000, 2568, "holes"),
    (1, 32, 3, 64, "same"), (1, 33, 3, 64, "same"), (1, 96, 2, 64, "uniform"), (1, 4096, 20000, 24, "skewed"),
    (1, 4097, 20000, 24, "skewed"), (3, 100001, 1000, 16, "skewed"), (1, 130, 9, 8200, "skewed"),
    (2, 33, 20, 20011, "uniform"), (1, 9000, 40, 16, "same"), (7, 3, 12, 2560, "uniform"),
]


@gpu
@pytest.mark.parametrize("tx", [F, B16], ids=["x32", "x16"])
@pytest.mark.parametrize("tE", [F, B16], ids=["E32", "E16"])
@pytest.mark.parametrize("B,T,vocab,d,kind", CASES)
def test_embed(B, T, vocab, d, kind, tE, tx):
    g = torch.Generator().manual_seed(d)
    E = torch.randn((vocab, d), generator=g).to(tE)
    ids = make_ids(B, T, vocab, kind)
    scale = 1.7
    known = (ids >= 0) & (ids < vocab)
    ref = E.double()[ids.long().clamp(0, vocab - 1)] * float(torch.tensor(scale)) * known[..., None]
    x = Guarded((B, T, d), tx)
    got = ttt.ttt_embed(guarded(E.cuda()), ids.cuda().contiguous(), scale=scale, x=x.t)
    torch.cuda.synchronize()
    x.check()
    assert_close(got, ref, (2 * U32 + 1.01 * half_step(tx)) * ref.abs(), "x")
    # the [B][T+1] ids of the layer, of which the last column is not this call's
    full = torch.cat([ids, torch.full((B, 1), 5, dtype=torch.int32)], 1).cuda()
    assert torch.equal(ttt.ttt_embed(E.cuda(), full[:, :T], scale=scale, dtype=tx), got)


@gpu
@pytest.mark.parametrize("tE", [F, B16], ids=["dE32", "dE16"])
@pytest.mark.parametrize("tx", [F, B16], ids=["dx32", "dx16"])
@pytest.mark.parametrize("B,T,vocab,d,kind", CASES)
def test_embed_grad(B, T, vocab, d, kind, tx, tE):
    g = torch.Generator().manual_seed(d + 1)
    dx = torch.randn((B, T, d), generator=g).to(tx)
    ids = make_ids(B, T, vocab, kind)
    flat = ids.reshape(-1)
    known = (flat >= 0) & (flat < vocab)
    scale = 0.75
    rows = dx.double().reshape(-1, d)
    at = flat.long()[known]
    ref = torch.zeros(vocab, d, dtype=torch.float64).index_add_(0, at, rows[known]) * scale
    mag = torch.zeros(vocab, d, dtype=torch.float64).index_add_(0, at, rows[known].abs()) * scale
    count = torch.bincount(at, minlength=vocab).double()
    adds = torch.minimum(count, 31 + torch.ceil(count / 256) + 9)[:, None] + 2
    bound = adds * U32 * mag
    dx_dev = dx.cuda()
    # rows of dx whose id is no row of the table are not read
    dx_dev.reshape(-1, d)[~known.cuda()] = float("nan")
    dx_dev = guarded(dx_dev)
    full = torch.cat([ids, torch.full((B, 1), 0, dtype=torch.int32)], 1).cuda()
    dE = Guarded((vocab, d), tE, fill=torch.full((vocab, d), float("nan")).to(tE))
    got = ttt.ttt_embed_grad(dx_dev, full[:, :T], vocab, scale=scale, dE=dE.t)
    torch.cuda.synchronize()
    dE.check()
    assert_close(got, ref, bound + half_step(tE) * (ref.abs() + bound), "dE")
    assert torch.equal(ttt.ttt_embed_grad(dx_dev, ids.cuda().contiguous(), vocab, scale=scale, dtype=tE), got)
    # added to what is there; rows that do not occur keep their bits
    old = torch.randn((vocab, d), generator=g).to(tE)
    if not bool(known.all()):
        old[count == 0] = float("nan")
    acc = Guarded((vocab, d), tE, fill=old)
    ttt.ttt_embed_grad(dx_dev, full[:, :T], vocab, scale=scale, dE=acc.t, accumulate=True)
    torch.cuda.synchronize()
    acc.check()
    hit = count > 0
    assert torch.equal(acc.t.cpu()[~hit].view(torch.uint8), old[~hit].contiguous().view(torch.uint8))
    want = (old.double() + ref)[hit]
    b = (bound + U32 * (old.double().abs() + mag))[hit]
    assert_close(acc.t[hit.cuda()], want, b + half_step(tE) * (want.abs() + b), "accumulated")


@gpu
def test_gradient_is_the_adjoint_and_follows_differences():
    """<embed(E), dx> = <E, embed_grad(dx)>, and along a random change of E the lookup's difference is the gradient's
    (the lookup is linear, so the difference has no error of its own)."""
    g = torch.Generator().manual_seed(3)
    vocab, d = 37, 48
    E, step = torch.randn((vocab, d), generator=g), torch.randn((vocab, d), generator=g)
    ids, dx = make_ids(3, 50, vocab, "holes"), torch.randn((3, 50, d), generator=g)
    dE = ttt.ttt_embed_grad(dx.cuda(), ids.cuda().contiguous(), vocab, scale=1.25).double().cpu()
    x = ttt.ttt_embed(E.cuda(), ids.cuda().contiguous(), scale=1.25).double().cpu()
    up = ttt.ttt_embed((E + step).cuda(), ids.cuda().contiguous(), scale=1.25).double().cpu()
    moved = (E + step).double() - E.double()
    mag = float((x * dx.double()).abs().sum() + (up * dx.double()).abs().sum())
    assert abs(float((x * dx.double()).sum()) - float((E.double() * dE).sum())) <= 80 * U32 * mag
    assert abs(float(((up - x) * dx.double()).sum()) - float((moved * dE).sum())) <= 80 * U32 * mag
    E64 = E.double().requires_grad_()
    known = (ids >= 0) & (ids < vocab)
    loss = (E64[ids.long().clamp(0, vocab - 1)] * known[..., None] * 1.25 * dx.double()).sum()
    auto = torch.autograd.grad(loss, E64)[0]
    assert_close(dE, auto, 80 * U32 * torch.full_like(auto, float(auto.abs().max()) + 1), "dE")


@gpu
def test_no_tokens():
    for shape in [(0,), (3, 0), (0, 4)]:
        ids = torch.empty(shape, dtype=torch.int32, device="cuda")
        E = torch.ones(2000, 64, device="cuda")
        assert ttt.ttt_embed(E, ids).shape == shape + (64,)
        dx = torch.empty(shape + (64,), device="cuda")
        assert bool((ttt.ttt_embed_grad(dx, ids, 2000) == 0).all())
        assert bool((ttt.ttt_embed_grad(dx, ids, 2000, dE=E, accumulate=True) == 1).all())


@gpu
def test_table_past_32_bit_offsets():
    """Rows whose byte (and element) offsets leave 32 bits."""
    vocab, d = 300001, 8192  # 2.46e9 elements
    E = torch.zeros((vocab, d), dtype=B16, device="cuda")
    E[-1] = torch.arange(d, device="cuda").to(B16)
    E[262144] = 3.0  # starts at element 2^31
    ids = torch.tensor([vocab - 1, 0, 262144, vocab - 1], dtype=torch.int32, device="cuda")
    x = ttt.ttt_embed(E, ids, scale=2.0)
    assert torch.equal(x[0], E[-1] * 2) and bool((x[1] == 0).all()) and bool((x[2] == 6).all())
    dx = torch.ones((4, d), dtype=B16, device="cuda")
    dE = ttt.ttt_embed_grad(dx, ids, vocab, dE=E)
    rows = dE.float().sum(1)
    want = torch.zeros(vocab, device="cuda")
    want[-1], want[0], want[262144] = 2 * d, d, d
    assert torch.equal(rows, want)


@gpu
@pytest.mark.parametrize("tx", [F, B16], ids=["x32", "x16"])
def test_more_than_the_caches_hold(tx):
    """Outputs over half a GiB, which are written past the caches, two rows at a time: an odd number of them."""
    vocab, d = 70001, 1032
    n = 600 * 2 ** 20 // (d * (4 if tx == F else 2)) | 1
    E = torch.randn((vocab, d), device="cuda").to(B16)
    ids = torch.randint(-1, vocab + 1, (n,), device="cuda").int()
    x = ttt.ttt_embed(E, ids, scale=3.0, dtype=tx)
    known = (ids >= 0) & (ids < vocab)
    want = (E[ids.long().clamp(0, vocab - 1)].float() * 3.0 * known[:, None]).to(tx)
    assert torch.equal(x, want)  # 3 e is exact in fp32, so both round the same number once


@gpu
@pytest.mark.parametrize("tE", [F, B16], ids=["dE32", "dE16"])
def test_gradient_of_a_table_past_the_caches(tE):
    """Over half a GiB of gradient, whose rows are written past the caches and dealt to the dies in runs: each row that
    occurs against 64 bits, and all others zero."""
    vocab, d, n = (70001, 2056, 6001) if tE == F else (70001, 4104, 6001)
    ids = make_ids(1, n, vocab, "skewed", seed=4)[0]
    g = torch.Generator().manual_seed(8)
    dx = torch.randn((n, d), generator=g).to(B16)
    dE = ttt.ttt_embed_grad(dx.cuda(), ids.cuda(), vocab, dE=torch.full((vocab, d), 7.0, dtype=tE, device="cuda"))
    rows, inverse, count = torch.unique(ids.long(), return_inverse=True, return_counts=True)
    ref = torch.zeros((len(rows), d), dtype=torch.float64).index_add_(0, inverse, dx.double())
    mag = torch.zeros((len(rows), d), dtype=torch.float64).index_add_(0, inverse, dx.double().abs())
    bound = (torch.minimum(count, 31 + torch.ceil(count / 256) + 9)[:, None] + 2) * U32 * mag
    assert_close(dE[rows.cuda()], ref, bound + half_step(tE) * (ref.abs() + bound), "dE")
    dE[rows.cuda()] = 0
    assert int(torch.count_nonzero(dE)) == 0


@gpu
def test_another_stream_and_graph_replays():
    vocab, d = 5000, 520
    ids = make_ids(2, 700, vocab, "skewed").cuda().contiguous()
    E = torch.randn((vocab, d), device="cuda")
    dx = torch.randn((2, 700, d), device="cuda")

    def step(stream=None):
        return [ttt.ttt_embed(E, ids, dtype=B16, stream=stream), ttt.ttt_embed_grad(dx, ids, vocab, stream=stream)]

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
        ids.copy_(make_ids(2, 700, vocab, "holes" if k % 2 else "same", seed=k).cuda())
        eager = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out)), k


def test_refusals():
    E, ids = torch.zeros(10, 64), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        ttt.ttt_embed(E, ids)
    with pytest.raises(ValueError, match=r"\[vocab\]"):
        ttt.ttt_embed(torch.zeros(10), ids)
    with pytest.raises(TypeError):
        ttt.ttt_embed(E.tolist(), ids)
    with pytest.raises(ValueError, match="int32"):
        ttt.ttt_embed_grad(torch.zeros(4, 64), ids.long(), 10)
    L = ttt.lib()

    def embed(E=1 << 30, Edt=0, vocab=10, d=64, ids=1 << 20, ld=8, B=2, T=8, scale=1.0, x=1 << 24, xdt=0):
        return L.ttt_embed(E, Edt, vocab, d, ids, ld, B, T, scale, x, xdt, None)

    assert embed(E=None) == -1 and embed(ids=None) == -1 and embed(x=None) == -1
    assert embed(Edt=3) == -3 and embed(xdt=-1) == -3
    assert embed(vocab=0) == -2 and embed(d=4) == -2 and embed(d=65537) == -2 and embed(ld=7) == -2
    assert embed(B=-1) == -2 and embed(T=-1) == -2 and embed(B=1 << 14, T=1 << 14, ld=1 << 14) == -2
    assert embed(scale=float("nan")) == -7 and embed(x=(1 << 24) + 2) == -7 and embed(ids=(1 << 20) + 2) == -7
    assert embed(x=1 << 30) == -7 and embed(x=1 << 20) == -7

    def grad(dx=1 << 30, ids=1 << 20, ld=8, vocab=10, d=64, dE=1 << 24, ws=1 << 27, nws=1 << 20, dt=0):
        return L.ttt_embed_grad(dx, dt, ids, ld, 2, 8, 1.0, vocab, d, dE, 0, 0, ws, nws, None)

    assert grad(dx=None) == -1 and grad(dE=None) == -1 and grad(ws=None) == -1
    assert grad(nws=100) == -2 and grad(vocab=-1) == -2 and grad(dt=2) == -3
    assert grad(dE=1 << 30) == -7 and grad(ws=1 << 24) == -7 and grad(ws=(1 << 27) + 8) == -7
    assert L.ttt_embed_grad_ws_bytes(1, 1, 1, 8, None) == -1


@gpu
def test_refusals_of_the_binding():
    E, ids = torch.zeros(10, 64, device="cuda"), torch.zeros((4, 6), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="2-D view"):
        ttt.ttt_embed(E, ids.t())
    with pytest.raises(ValueError, match="2-D view"):
        ttt.ttt_embed(E, ids[:, ::2])
    with pytest.raises(ValueError, match="shape"):
        ttt.ttt_embed(E, ids, x=torch.zeros(24, 64, device="cuda"))
    with pytest.raises(ValueError, match="dx must be"):
        ttt.ttt_embed_grad(torch.zeros(4, 64, device="cuda"), ids, 10)
    with pytest.raises(ValueError, match="dtype must be"):
        ttt.ttt_embed(E, ids, dtype=torch.float16)
    with pytest.raises(ValueError, match="dtype must be"):
        ttt.ttt_embed_grad(torch.zeros(4, 6, 64, device="cuda"), ids, 10, dtype=torch.int32)
    with pytest.raises(ValueError, match="dE must be given"):
        ttt.ttt_embed_grad(torch.zeros(4, 6, 64, device="cuda"), ids, 10, accumulate=True)
    with pytest.raises(ValueError, match="shape"):
        ttt.ttt_embed_grad(torch.zeros(4, 6, 64, device="cuda"), ids, 10, dE=torch.zeros(9, 64, device="cuda"))


@gpu
def test_more_rows_than_a_grid_side_counts():
    """2^22 + 3 rows of 8192: at 1024 threads a row they pass 2^32."""
    n, d = 2 ** 22 + 3, 8192
    E = torch.arange(1, 4, device="cuda", dtype=torch.float32)[:, None].expand(3, d).contiguous().to(B16)
    ids = (torch.arange(n, device="cuda") % 3).int()
    x = ttt.ttt_embed(E, ids)
    assert torch.equal(x[:, 0], E[:, 0][ids.long()]) and torch.equal(x[-5:], E[ids[-5:].long()])
    assert torch.equal(x[:, -1], x[:, 0])


@gpu
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,d", [(2 ** 17 + 5, 72), (2 ** 22, 8), (2 ** 22 - 17, 9)])
def test_one_id_in_a_long_batch(n, d, accumulate):
    """A padding id that takes most of a batch: the pieces of 32 tokens are summed in fp32 (31 additions), eight
    pieces again (7), and those sums in fp64, so the error's bound does not grow with the tokens. All gradients are the
    same number, chosen so that a running fp32 sum of the pieces would lose up to half of a piece's last place with each
    of them, always downwards."""
    value = (1 + 501 * 2.0 ** -20) / 32
    dx = torch.full((n, d), value, device="cuda")
    ids = torch.full((n,), 1, dtype=torch.int32, device="cuda")
    ids[::1000] = 0
    dE = torch.ones((3, d), device="cuda") if accumulate else None
    got = ttt.ttt_embed_grad(dx, ids, 3, dE=dE, accumulate=accumulate)
    count = torch.bincount(ids.long(), minlength=3).double().cpu()[:, None]
    ref = count * value + (1.0 if accumulate else 0.0)
    # 31 + 7 additions, and a rounding each of the joined sum, its scaling and the accumulation
    assert_close(got, ref.expand(3, d), (41 * U32 * ref).expand(3, d), "dE")


def test_sizes_past_32_bits_are_refused():
    """Sizes that a 32-bit int would hold the low bits of only (meta tensors: no memory behind them)."""
    def ids(*shape):
        return torch.empty(shape, dtype=torch.int32, device="meta")

    def dx(*shape):
        return torch.empty(shape, device="meta")

    big = 2 ** 32 + 64
    for call in (lambda: ttt.ttt_embed(dx(big, 64), ids(4)), lambda: ttt.ttt_embed(dx(10, big), ids(4)),
                 lambda: ttt.ttt_embed_grad(dx(4, 64), ids(4), big),
                 lambda: ttt.ttt_embed_grad(dx(4, 64), ids(4), 64 - 2 ** 32),
                 lambda: ttt.ttt_embed_grad(dx(4, big), ids(4), 10),
                 lambda: ttt.ttt_embed_grad(dx(big, 64), ids(big), 10),
                 lambda: ttt.ttt_embed_grad(dx(2, big, 64), ids(2, big + 1)[:, :big], 10)):
        with pytest.raises(ValueError, match=r"2\^31"):
            call()


@gpu
@pytest.mark.parametrize("kind", ["skewed", "holes"])
@pytest.mark.parametrize("T,vocab", [(2999, 8192), (3000, 8192), (3001, 8192), (4095, 8191), (4096, 8191), (4097, 8191),
                                     (4096, 8192), (3001, 151936), (1025, 8191), (1024, 8192)])
def test_gradient_where_the_sort_changes(T, vocab, kind):
    """One workgroup sorts up to 4096 tokens of a table of up to 8191 rows, 3000 of larger ones; more go by tiles."""
    test_embed_grad(1, T, vocab, 24, kind, F, F)

"""The calls on many tensors with the lists read in Python: the same bits as with the native reader."""
import pytest
import torch

import chunk_wise_weight_amd as ttt
from chunk_wise_weight_amd import binding

pytestmark = pytest.mark.gpu


def test_lists_read_in_python(monkeypatch):
    gen = torch.Generator().manual_seed(1)
    sizes = [(1,), (300,), (0,), (33, 40), (5000,)]

    def results():
        torch.manual_seed(0)
        gen.manual_seed(1)
        w, g, m = ([torch.randn(s, generator=gen).cuda() for s in sizes] for _ in range(3))
        g[3] = g[3].bfloat16()
        v = [t * t for t in m]
        c = [t.bfloat16() for t in w]
        m8, v8 = ([torch.zeros(s, dtype=torch.uint8, device="cuda") for s in sizes] for _ in range(2))
        tops = [torch.zeros((2, -(-t.numel() // 256)), dtype=torch.int16, device="cuda") for t in w]
        norm = ttt.ttt_grad_norm(g)
        out = [torch.empty_like(t) for t in g]
        again = ttt.ttt_clip_grads(g, 0.5, out=out)
        ttt.ttt_adamw(w, out, m, v, 3, 1e-2, copies=c, norm=norm, tau=0.25)
        ttt.ttt_adamw(w, g, m8, v8, 1, 1e-2, tops=tops, seed=7)
        return [norm, again, *out, *w, *m, *v, *c, *m8, *v8, *tops, *ttt.ttt_adamw_values(m8, tops, 1)]

    want = results()
    monkeypatch.setattr(binding, "_read", binding._read_python)
    for a, b in zip(results(), want):
        assert torch.equal(a, b)
    x, side = torch.ones(4, device="cuda"), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = ttt.ttt_grad_norm([x], stream=side)
    side.synchronize()
    assert float(norm) == 2.0
    with pytest.raises(ValueError, match="contiguous"):
        ttt.ttt_grad_norm([torch.zeros(3, 4, device="cuda").T])
    with pytest.raises(ValueError, match="device tensors"):
        ttt.ttt_grad_norm([x, torch.zeros(3)])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ttt.ttt_grad_norm([x.double()])

"""Helpers of the tests of the operators around the layer: guarded arrays and the formulas in 64 bits."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


class Guarded:
    """A tensor that starts on an odd element of a larger buffer, with marks on both sides of it."""

    MARK = 77.0

    def __init__(self, shape, dtype, off=3, device="cuda", fill=None):
        n = 1
        for s in shape:
            n *= s
        self.buf = torch.full((n + off + 64,), self.MARK, dtype=dtype, device=device)
        self.off, self.n = off, n
        self.t = self.buf[off:off + n].view(shape)
        if fill is not None:
            self.t.copy_(fill)

    def check(self):
        assert bool((self.buf[:self.off] == self.MARK).all()), "written before the array"
        assert bool((self.buf[self.off + self.n:] == self.MARK).all()), "written past the array"


def guarded(t, off=3):
    """t's values in a guarded array."""
    return Guarded(tuple(t.shape), t.dtype, off, t.device, t).t


def rms64(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def assert_close(got, ref, bound, what):
    """|got - ref| <= bound element by element (both finite)."""
    got = got.double().cpu()
    err = (got - ref).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = int(torch.where(bad.reshape(-1))[0][0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} past the bound; first at {i}: got "
                             f"{got.reshape(-1)[i].item()!r}, want {ref.reshape(-1)[i].item()!r}, bound "
                             f"{bound.expand_as(ref).reshape(-1)[i].item():.3g}")

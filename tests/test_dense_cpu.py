"""Refusals of the plain layers' and the step's entry points that need no GPU: every one comes before any device work."""
import ctypes

import pytest
import torch

import chunk_wise_weight_amd as ttt

NULL, SHAPE, DTYPE, ARG = -1, -2, -3, -7


def P(v):
    return ctypes.c_void_p(v)


def linear(x=0x1000, W=0x200000, dt=1, bias=0, act=0, scale=1.0, res=0, rows=4, n=8, out=16, pre=0, y=0x400000, y_dt=1,
           ws=0x800000, nws=1 << 20):
    return ttt.lib().ttt_linear(P(x), P(W), dt, P(bias), act, scale, P(res), rows, n, out, P(pre), P(y), y_dt, P(ws),
                                nws, None)


def gated(x=0x1000, Wg=0x200000, Wu=0x300000, dt=1, bg=0, bu=0, act=1, rows=4, n=8, f=16, g=0, u=0, z=0x400000,
          ws=0x800000, nws=1 << 20):
    return ttt.lib().ttt_gated(P(x), P(Wg), P(Wu), dt, P(bg), P(bu), act, rows, n, f, P(g), P(u), P(z), P(ws), nws, None)


def linear_grad(dy=0x1000, y_dt=1, x=0x100000, W=0x200000, dt=1, pre=0, act=0, scale=1.0, rows=4, n=8, out=16,
                dx=0x400000, dW=0x500000, db=0x600000, acc=0, ws=0x800000, nws=1 << 20):
    return ttt.lib().ttt_linear_grad(P(dy), y_dt, P(x), P(W), dt, P(pre), act, scale, rows, n, out, P(dx), P(dW), P(db),
                                     acc, P(ws), nws, None)


def gated_grad(dz=0x1000, x=0x100000, Wg=0x200000, Wu=0x300000, dt=1, g=0x400000, u=0x500000, act=1, rows=4, n=8, f=16,
               dx=0x600000, dWg=0x700000, dWu=0x800000, dbg=0, dbu=0, acc=0, ws=0xa00000, nws=1 << 20):
    return ttt.lib().ttt_gated_grad(P(dz), P(x), P(Wg), P(Wu), dt, P(g), P(u), act, rows, n, f, P(dx), P(dWg), P(dWu),
                                    P(dbg), P(dbu), acc, P(ws), nws, None)


@pytest.mark.parametrize("call,code", [
    (lambda: linear(x=0), NULL), (lambda: linear(W=0), NULL), (lambda: linear(y=0), NULL),
    (lambda: linear(dt=2), DTYPE), (lambda: linear(y_dt=5), DTYPE), (lambda: linear(dt=0, y_dt=1), DTYPE),
    (lambda: linear(rows=-1), SHAPE), (lambda: linear(rows=2 ** 31), SHAPE), (lambda: linear(n=0), SHAPE),
    (lambda: linear(out=(1 << 20) + 1), SHAPE), (lambda: linear(act=4), ARG), (lambda: linear(act=-1), ARG),
    (lambda: linear(scale=float("nan")), ARG), (lambda: linear(x=0x1001), ARG), (lambda: linear(y=0x1000), ARG),
    (lambda: linear(y=0x400001), ARG), (lambda: linear(pre=0x400000), ARG), (lambda: linear(res=0x400002), ARG),
    (lambda: gated(Wu=0), NULL), (lambda: gated(bg=0x1400000), NULL), (lambda: gated(g=0x1400000), NULL),
    (lambda: gated(act=0), ARG), (lambda: gated(dt=3), DTYPE), (lambda: gated(n=-3), SHAPE),
    (lambda: gated(z=0x200010), ARG), (lambda: gated(g=0x1400000, u=0x1400010), ARG),
    (lambda: linear_grad(dy=0), NULL), (lambda: linear_grad(x=0), NULL), (lambda: linear_grad(W=0), NULL),
    (lambda: linear_grad(act=1), NULL), (lambda: linear_grad(ws=0), NULL), (lambda: linear_grad(ws=0x800008), ARG),
    (lambda: linear_grad(nws=16), SHAPE), (lambda: linear_grad(dW=0x200000), ARG), (lambda: linear_grad(dx=0x800000), ARG),
    (lambda: linear_grad(dt=0, y_dt=1), DTYPE), (lambda: linear_grad(scale=float("inf")), ARG),
    (lambda: gated_grad(g=0), NULL), (lambda: gated_grad(dWu=0), NULL), (lambda: gated_grad(dbg=0xc00000), NULL),
    (lambda: gated_grad(act=7), ARG), (lambda: gated_grad(rows=-2), SHAPE), (lambda: gated_grad(dx=0x1004), ARG),
    (lambda: gated_grad(nws=0), SHAPE),
])
def test_refusals(call, code):
    assert call() == code
    assert ttt.ttt_last_error()


def adamw(n=2, w=(0x1000, 0x2000), g=(0x3000, 0x4000), m=(0x5000, 0x6000), v=(0x7000, 0x8000), tops=None, copies=None,
          numel=(4, 4), bits=32, step=1, step_dev=0, lr=1e-3, lr_dev=0, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, norm=0,
          tau=1.0, w_dt=(0, 0), g_dt=(0, 0)):
    def ptrs(a):
        return None if a is None else (ctypes.c_void_p * len(a))(*a)

    def ints(a, t):
        return None if a is None else (t * len(a))(*a)

    return ttt.lib().ttt_adamw(ptrs(w), ints(w_dt, ctypes.c_int32), ptrs(g), ints(g_dt, ctypes.c_int32), ptrs(m),
                               ptrs(v), bits, ptrs(tops), ptrs(copies), ints(numel, ctypes.c_int64), n, step,
                               P(step_dev), lr, P(lr_dev), b1, b2, eps, wd, P(norm), tau, 0, None)


@pytest.mark.parametrize("call,code", [
    (lambda: adamw(n=-1), SHAPE), (lambda: adamw(n=2 ** 20 + 1), SHAPE), (lambda: adamw(numel=None), NULL),
    (lambda: adamw(numel=(4, -1)), SHAPE), (lambda: adamw(numel=(2 ** 40, 2 ** 40)), SHAPE), (lambda: adamw(w=None), NULL),
    (lambda: adamw(v=None), NULL), (lambda: adamw(w_dt=None), NULL), (lambda: adamw(bits=16), ARG),
    (lambda: adamw(bits=8), NULL), (lambda: adamw(step=0), ARG), (lambda: adamw(b1=1.0), ARG), (lambda: adamw(b2=-0.1), ARG),
    (lambda: adamw(b1=float("nan")), ARG), (lambda: adamw(eps=-1.0), ARG), (lambda: adamw(wd=float("inf")), ARG),
    (lambda: adamw(lr=float("nan")), ARG), (lambda: adamw(norm=0x9000, tau=0.0), ARG),
    (lambda: adamw(norm=0x9000, tau=float("nan")), ARG), (lambda: adamw(w_dt=(0, 2)), DTYPE),
    (lambda: adamw(g=(0, 0x4000)), NULL), (lambda: adamw(m=(0x5002, 0x6000)), ARG), (lambda: adamw(w=(0x1000, 0x1008)), ARG),
    (lambda: adamw(m=(0x3000, 0x6000)), ARG), (lambda: adamw(copies=(0x1000, 0)), ARG), (lambda: adamw(norm=0x1004), ARG),
    (lambda: adamw(step_dev=0x9004), ARG), (lambda: adamw(bits=8, tops=(0xa001, 0xb000)), ARG),
    (lambda: adamw(bits=8, tops=(0xa000, 0xa002)), ARG),
])
def test_refusals_of_the_step(call, code):
    assert call() == code
    assert ttt.ttt_last_error()


def test_refusals_of_the_values():
    L = ttt.lib()
    one, size = (ctypes.c_void_p * 1)(0x1000), (ctypes.c_int64 * 1)(300)
    tops, out = (ctypes.c_void_p * 1)(0x2000), (ctypes.c_void_p * 1)(0x3000)
    assert L.ttt_adamw_values(one, tops, 3, out, size, 1, None) == ARG
    assert L.ttt_adamw_values(one, None, 1, out, size, 1, None) == NULL
    assert L.ttt_adamw_values(one, tops, 1, (ctypes.c_void_p * 1)(0x2004), size, 1, None) == ARG
    assert L.ttt_adamw_values(one, tops, 1, (ctypes.c_void_p * 1)(0x3002), size, 1, None) == ARG
    assert L.ttt_adamw_values(one, tops, 1, out, size, -1, None) == SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_a_device():
    assert linear() == gated() == linear_grad() == gated_grad() == adamw() == -6
    assert adamw(bits=8, tops=(0xa000, 0xb000)) == -6


def test_workspace_queries():
    n = ctypes.c_size_t()
    L = ttt.lib()
    q = L.ttt_linear_grad_ws_bytes
    assert q(1000, 64, 64, 1, 1, 0, ctypes.byref(n)) == 0
    small = n.value
    # q is made with an activation, or from an fp32 dy
    for y_dt, act in ((0, 0), (1, 2), (0, 2)):
        assert q(1000, 64, 64, 1, y_dt, act, ctypes.byref(n)) == 0 and n.value >= small + 1000 * 64 * 2
    assert q(100, 64, 64, 0, 1, 0, ctypes.byref(n)) == DTYPE
    assert q(100, 64, 64, 1, 1, 9, ctypes.byref(n)) == ARG
    for q in (L.ttt_linear_ws_bytes, L.ttt_gated_ws_bytes, L.ttt_gated_grad_ws_bytes):
        assert q(100, 64, 64, 1, ctypes.byref(n)) == 0
        assert q(100, 64, 64, 1, None) == NULL
        assert q(100, 0, 64, 1, ctypes.byref(n)) == SHAPE
        assert q(100, 64, 64, 9, ctypes.byref(n)) == DTYPE


def test_refusals_of_the_binding():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="device tensor"):
        ttt.ttt_linear(x, w)
    with pytest.raises(ValueError, match=r"\[out\]\[8\]"):
        ttt.ttt_linear(x, torch.zeros(8, 6))
    with pytest.raises(TypeError, match="w must be a tensor"):
        ttt.ttt_linear(x, None)
    with pytest.raises(ValueError, match="device tensor"):
        ttt.ttt_gated(x, w, w)
    with pytest.raises(ValueError, match="device tensors"):
        ttt.ttt_adamw([x], [x], [x], [x], 1, 1e-3)
    with pytest.raises(ValueError, match="one tensor per parameter|device"):
        ttt.ttt_adamw([x], [], [x], [x], 1, 1e-3)
    with pytest.raises(ValueError, match="tops must be given"):
        ttt.ttt_adamw([x], [x], [x.to(torch.uint8)], [x.to(torch.uint8)], 1, 1e-3)
    with pytest.raises(ValueError, match="seed"):
        ttt.ttt_adamw([x], [x], [x], [x], 1, 1e-3, seed=-1)

"""Python binding of libttt.so: the C ABI's entry points under the same names.

Argument marshalling only: tensors are turned into device pointers and sizes,
and torch's current HIP stream is passed along. Every step of the
computation runs in the library's HIP kernels; there is no fallback path, and
a missing or unloadable library raises.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from functools import lru_cache
from operator import attrgetter
from typing import Dict, List, NamedTuple, Optional, Tuple

import torch  # loads the HIP runtime the library binds to (same libamdhip64 soname)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libttt.so")

TTT_F32, TTT_BF16 = 0, 1
ERRORS = {-1: "TTT_E_NULL", -2: "TTT_E_SHAPE", -3: "TTT_E_DTYPE", -4: "TTT_E_NOMEM", -5: "TTT_E_HIP",
          -6: "TTT_E_NODEV", -7: "TTT_E_ARG"}
EXPORTS = ("ttt_init", "ttt_forward_chunked", "ttt_forward_docs", "ttt_reset", "ttt_destroy", "ttt_last_error",
           "ttt_set_group_chunks", "ttt_set_clip", "ttt_set_target_conv", "ttt_plan", "ttt_set_profiling", "ttt_phase_times",
           "ttt_workspace_bytes", "ttt_set_output_f32", "ttt_state_delta", "ttt_forward_chunked_noalloc",
           "ttt_norm_pre", "ttt_norm_post", "ttt_norm_ws_bytes", "ttt_norm_pre_grad", "ttt_norm_post_grad",
           "ttt_embed", "ttt_embed_grad_ws_bytes", "ttt_embed_grad", "ttt_grad_ws_bytes", "ttt_grad_norm",
           "ttt_clip_grads")

_lib = None


class TTTError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where}: {ERRORS.get(code, code)}: {msg}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libttt.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m chunk_wise_weight_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.ttt_init.argtypes = [ctypes.POINTER(vp), vp, vp, vp, i32, i32, i32, f32, i32, i32, vp]
    L.ttt_init.restype = i32
    L.ttt_forward_chunked.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp]
    L.ttt_forward_chunked.restype = i32
    L.ttt_reset.argtypes = [vp, i32, vp]
    L.ttt_reset.restype = i32
    L.ttt_destroy.argtypes = [vp]
    L.ttt_destroy.restype = None
    L.ttt_last_error.argtypes = []
    L.ttt_last_error.restype = ctypes.c_char_p
    L.ttt_set_group_chunks.argtypes = [vp, i32]
    L.ttt_set_group_chunks.restype = i32
    L.ttt_set_clip.argtypes = [vp, f32]
    L.ttt_set_clip.restype = i32
    L.ttt_set_target_conv.argtypes = [vp, vp, i32, vp, vp]
    L.ttt_set_target_conv.restype = i32
    ip = ctypes.POINTER(i32)
    L.ttt_forward_docs.argtypes = [vp, vp, vp, vp, i32, i32, i32, ip, ip, vp, vp, vp]
    L.ttt_forward_docs.restype = i32
    L.ttt_plan.argtypes = [i32, i32, i32, ip, ip, ip, ip]
    L.ttt_plan.restype = i32
    L.ttt_set_profiling.argtypes = [vp, i32]
    L.ttt_set_profiling.restype = i32
    L.ttt_phase_times.argtypes = [vp, ctypes.POINTER(f32), i32]
    L.ttt_phase_times.restype = i32
    L.ttt_workspace_bytes.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t)]
    L.ttt_workspace_bytes.restype = i32
    L.ttt_set_output_f32.argtypes = [vp, i32]
    L.ttt_set_output_f32.restype = i32
    L.ttt_state_delta.argtypes = [vp, vp, i32, vp]
    L.ttt_state_delta.restype = i32
    L.ttt_forward_chunked_noalloc.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp]
    L.ttt_forward_chunked_noalloc.restype = i32
    i64, sz = ctypes.c_int64, ctypes.c_size_t
    L.ttt_norm_pre.argtypes = [vp, i32, vp, i32, f32, i64, i32, vp, i32, vp]
    L.ttt_norm_post.argtypes = [vp, i32, vp, i32, vp, vp, i32, vp, i32, f32, f32, f32, i64, i32, vp, vp, i32, vp]
    L.ttt_norm_ws_bytes.argtypes = [i64, i32, ctypes.POINTER(sz)]
    L.ttt_norm_pre_grad.argtypes = [vp, i32, vp, i32, vp, i32, vp, f32, i64, i32, vp, vp, vp, sz, vp]
    L.ttt_norm_post_grad.argtypes = [vp, vp, i32, vp, i32, vp, i32, vp, vp, i32, vp, i32, f32, f32, f32, i64, i32, vp,
                                     vp, vp, vp, vp, vp, sz, vp]
    L.ttt_embed.argtypes = [vp, i32, i32, i32, vp, i64, i32, i32, f32, vp, i32, vp]
    L.ttt_embed_grad_ws_bytes.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    L.ttt_embed_grad.argtypes = [vp, i32, vp, i64, i32, i32, f32, i32, i32, vp, i32, i32, vp, sz, vp]
    L.ttt_grad_ws_bytes.argtypes = [i32, ctypes.POINTER(sz)]
    L.ttt_grad_norm.argtypes = [vp, vp, vp, i32, vp, vp, sz, vp]
    L.ttt_clip_grads.argtypes = [vp, vp, vp, i32, f32, vp, vp, vp, sz, vp]
    for fn in (L.ttt_norm_pre, L.ttt_norm_post, L.ttt_norm_ws_bytes, L.ttt_norm_pre_grad, L.ttt_norm_post_grad,
               L.ttt_embed, L.ttt_embed_grad_ws_bytes, L.ttt_embed_grad, L.ttt_grad_ws_bytes, L.ttt_grad_norm,
               L.ttt_clip_grads):
        fn.restype = i32
    _lib = L
    return L


def ttt_last_error() -> str:
    return lib().ttt_last_error().decode()


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise TTTError(rc, where, ttt_last_error())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _dev(t: torch.Tensor, name: str, dtype=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


class Handle:
    """An initialised layer (library handle) and the shapes it was made with."""

    def __init__(self, ptr: ctypes.c_void_p, d: int, f: int, C: int, eta: float, dtype: torch.dtype,
                 max_batch: int):
        self._ptr = ptr
        self.d, self.f, self.C, self.eta, self.dtype, self.max_batch = d, f, C, eta, dtype, max_batch
        self.y_dtype = dtype  # the dtype forward calls write y in

    @property
    def ptr(self) -> ctypes.c_void_p:
        if not self._ptr:
            raise RuntimeError("handle already destroyed")
        return self._ptr

    def __del__(self):
        try:
            ttt_destroy(self)
        except Exception:
            pass


def ttt_init(W_up: torch.Tensor, W_gate: torch.Tensor, W_down0: torch.Tensor, C: int, eta: float,
             max_batch: int = 1, stream=None) -> Handle:
    """W_up, W_gate [f][d]; W_down0 [d][f]; float32 or bfloat16 (all the same)."""
    dt = W_up.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError("weights must be float32 or bfloat16")
    for t, n in ((W_up, "W_up"), (W_gate, "W_gate"), (W_down0, "W_down0")):
        _dev(t, n, dt)
        if t.dim() != 2:
            raise ValueError(f"{n} must be 2-D")
    f, d = W_up.shape
    h = ctypes.c_void_p()
    _check(lib().ttt_init(ctypes.byref(h), _ptr(W_up), _ptr(W_gate), _ptr(W_down0), d, f, int(C), float(eta),
                          TTT_BF16 if dt == torch.bfloat16 else TTT_F32, int(max_batch), _stream(stream)),
           "ttt_init")
    if tuple(W_gate.shape) != (f, d) or tuple(W_down0.shape) != (d, f):
        ttt_destroy(Handle(h, d, f, C, eta, dt, max_batch))
        raise ValueError("shapes must be W_up, W_gate [f][d] and W_down0 [d][f]")
    return Handle(h, d, f, int(C), float(eta), dt, int(max_batch))


def _forward_args(h, x, ids, E_tgt, y, W_final, want_W_final):
    _dev(x, "x", h.dtype)
    _dev(ids, "ids", torch.int32)
    _dev(E_tgt, "E_tgt", h.dtype)
    if x.dim() != 3 or ids.dim() != 2 or E_tgt.dim() != 2:
        raise ValueError("x must be [B][T][d], ids [B][T+1], E_tgt [vocab][d]")
    B, T, d = x.shape
    if tuple(ids.shape) != (B, T + 1) or d != h.d or E_tgt.shape[1] != h.d:
        raise ValueError("shape mismatch among x, ids, E_tgt and the handle")
    if y is None:
        y = torch.empty((B, T, d), dtype=h.y_dtype, device=x.device)
    else:
        _dev(y, "y", h.y_dtype)
        if tuple(y.shape) != (B, T, d):
            raise ValueError("y must be [B][T][d]")
    if W_final is None and want_W_final:
        W_final = torch.empty((B, h.d, h.f), dtype=torch.float32, device=x.device)
    if W_final is not None:
        _dev(W_final, "W_final", torch.float32)
        if tuple(W_final.shape) != (B, h.d, h.f):
            raise ValueError("W_final must be [B][d][f]")
    return B, T, y, W_final



def ttt_forward_chunked(h: Handle, x: torch.Tensor, ids: torch.Tensor, E_tgt: torch.Tensor,
                        y: Optional[torch.Tensor] = None, W_final: Optional[torch.Tensor] = None,
                        want_W_final: bool = False, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """x [B][T][d], ids [B][T+1] int32, E_tgt [vocab][d] -> (y [B][T][d], W_final [B][d][f] fp32 or None)."""
    B, T, y, W_final = _forward_args(h, x, ids, E_tgt, y, W_final, want_W_final)
    _check(lib().ttt_forward_chunked(h.ptr, _ptr(x), _ptr(ids), _ptr(E_tgt), int(E_tgt.shape[0]), int(B), int(T),
                                     _ptr(y), _ptr(W_final), _stream(stream)), "ttt_forward_chunked")
    return y, W_final


NOALLOC_WORKSPACE_BYTES = 64 << 20  # TTT_NOALLOC_WORKSPACE_BYTES in include/ttt.h


def ttt_forward_chunked_noalloc(h: Handle, x: torch.Tensor, ids: torch.Tensor, E_tgt: torch.Tensor,
                                y: torch.Tensor, W_final: Optional[torch.Tensor] = None,
                                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """ttt_forward_chunked with the library's fixed workspace: the call allocates nothing on the device.
    y (and W_final, if wanted) must be given."""
    if y is None:
        raise ValueError("y must be given (the call allocates nothing)")
    B, T, y, W_final = _forward_args(h, x, ids, E_tgt, y, W_final, False)
    _check(lib().ttt_forward_chunked_noalloc(h.ptr, _ptr(x), _ptr(ids), _ptr(E_tgt), int(E_tgt.shape[0]), int(B),
                                             int(T), _ptr(y), _ptr(W_final), _stream(stream)),
           "ttt_forward_chunked_noalloc")
    return y, W_final


def ttt_forward_docs(h: Handle, x: torch.Tensor, ids: torch.Tensor, E_tgt: torch.Tensor, doc_starts,
                     y: Optional[torch.Tensor] = None, W_final: Optional[torch.Tensor] = None,
                     want_W_final: bool = False, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Packed documents: doc_starts[b] lists the positions in (0, T) where a new
    document starts in sequence b (the state returns to W_down0 there)."""
    B, T, y, W_final = _forward_args(h, x, ids, E_tgt, y, W_final, want_W_final)
    if len(doc_starts) != B:
        raise ValueError("doc_starts needs one list per sequence")
    counts = (ctypes.c_int32 * max(B, 1))(*[len(s) for s in doc_starts])
    flat = [int(p) for s in doc_starts for p in s]
    starts = (ctypes.c_int32 * max(len(flat), 1))(*flat)
    _check(lib().ttt_forward_docs(h.ptr, _ptr(x), _ptr(ids), _ptr(E_tgt), int(E_tgt.shape[0]), int(B), int(T),
                                  starts, counts, _ptr(y), _ptr(W_final), _stream(stream)), "ttt_forward_docs")
    return y, W_final

def ttt_reset(h: Handle, b: int = -1, stream=None) -> None:
    _check(lib().ttt_reset(h.ptr, int(b), _stream(stream)), "ttt_reset")


def ttt_destroy(h: Handle) -> None:
    if h._ptr:
        lib().ttt_destroy(h._ptr)
        h._ptr = None


def ttt_set_group_chunks(h: Handle, G: int) -> None:
    _check(lib().ttt_set_group_chunks(h.ptr, int(G)), "ttt_set_group_chunks")


def ttt_set_clip(h: Handle, tau: float) -> None:
    """Frobenius clipping of each chunk update at threshold tau (0 or inf: off)."""
    _check(lib().ttt_set_clip(h.ptr, float(tau)), "ttt_set_clip")


def ttt_set_target_conv(h: Handle, conv_w=None, W_target=None, stream=None) -> None:
    """The general target Conv1D(X0) W_target: conv_w [K][d], W_target [d][d]
    (device tensors of the handle's dtype). conv_w None restores the next-token target."""
    if conv_w is None:
        _check(lib().ttt_set_target_conv(h.ptr, None, 0, None, _stream(stream)), "ttt_set_target_conv")
        return
    cw = conv_w.contiguous()
    wt = W_target.contiguous()
    _dev(cw, "conv_w", h.dtype)
    _dev(wt, "W_target", h.dtype)
    if cw.dim() != 2 or cw.shape[1] != h.d or tuple(wt.shape) != (h.d, h.d):
        raise ValueError("shapes must be conv_w [K][d] and W_target [d][d]")
    _check(lib().ttt_set_target_conv(h.ptr, _ptr(cw), int(cw.shape[0]), _ptr(wt), _stream(stream)),
           "ttt_set_target_conv")


def ttt_plan(T: int, C: int, G: int = 0) -> Dict[str, int]:
    """Host-only: the group layout a call with T tokens and chunk C uses."""
    g, L, n, tp = (ctypes.c_int() for _ in range(4))
    _check(lib().ttt_plan(int(T), int(C), int(G), ctypes.byref(g), ctypes.byref(L), ctypes.byref(n),
                          ctypes.byref(tp)), "ttt_plan")
    return {"G": g.value, "L": L.value, "ngroups": n.value, "T_pad": tp.value}


def ttt_state_delta(h: Handle, B: Optional[int] = None, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """D = W - W_down0 of sequences 0 .. B-1 (the change since each last reset), [B][d][f] float32."""
    B = h.max_batch if B is None else int(B)
    if out is None:
        out = torch.empty((B, h.d, h.f), dtype=torch.float32, device="cuda")
    _dev(out, "out", torch.float32)
    if tuple(out.shape) != (B, h.d, h.f):
        raise ValueError("out must be [B][d][f]")
    _check(lib().ttt_state_delta(h.ptr, _ptr(out), B, _stream(stream)), "ttt_state_delta")
    return out


def ttt_set_output_f32(h: Handle, on: bool = True) -> None:
    """On a bfloat16 handle, later forward calls write y as float32 (no final rounding to bf16)."""
    _check(lib().ttt_set_output_f32(h.ptr, 1 if on else 0), "ttt_set_output_f32")
    h.y_dtype = torch.float32 if (on or h.dtype == torch.float32) else h.dtype


def ttt_set_profiling(h: Handle, on: bool = True) -> None:
    _check(lib().ttt_set_profiling(h.ptr, 1 if on else 0), "ttt_set_profiling")


PHASES = ("gather", "up_gate_swiglu", "clip_factors", "update_snapshots", "group_scores", "output", "final_copy")


def ttt_phase_times(h: Handle) -> List[float]:
    """Milliseconds per phase, the mean per forward call over the profiled calls since the previous read
    (waits for them)."""
    buf = (ctypes.c_float * len(PHASES))()
    _check(lib().ttt_phase_times(h.ptr, buf, len(PHASES)), "ttt_phase_times")
    return list(buf)


def ttt_workspace_bytes(h: Handle) -> int:
    n = ctypes.c_size_t()
    _check(lib().ttt_workspace_bytes(h.ptr, ctypes.byref(n)), "ttt_workspace_bytes")
    return n.value


# ---- the operators around the layer ----
#
# They take no handle. Tensors must be contiguous and on the current device; an
# output that is not given is allocated. With `stream` the work, and the
# outputs made here, belong to that stream, as under torch.cuda.stream(stream);
# what the tensors hold must be ready on it. They record no autograd graph:
# each gradient is a call of its own. Nor does autograd see what a call writes
# into a tensor it was given (no version is counted), so one that a graph has
# saved for its backward must not be given for an output.

_DT = {torch.float32: TTT_F32, torch.bfloat16: TTT_BF16}
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2


# the current stream's handle without a Stream object around it (2.6 us less on a call of about 10)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


class _Call:
    """The stream and device of one call, and the tensors it was given."""

    __slots__ = ("device", "stream", "where")

    def __init__(self, where: torch.device, stream):
        # no device tensor exists before torch has initialised the device
        self.device = torch.cuda.current_device() if torch.cuda.is_initialized() else -1
        self.stream = stream
        if stream is not None and stream.device.index != self.device:
            raise ValueError("stream must be on the current device")
        self.where = where

    def arg(self, t: Optional[torch.Tensor], name: str, dtype=None, shape=None) -> Optional[int]:
        """A tensor's address (None for None), after its checks."""
        if t is None:
            return None
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
        if t.dtype not in _DT:
            raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.get_device() != self.device or self.device < 0:  # -1: a host tensor
            raise ValueError(f"{name} must be {'on the current device' if t.is_cuda else 'a device tensor'}")
        if self.stream is not None:
            t.record_stream(self.stream)
        return t.data_ptr()

    def like(self, t: torch.Tensor, dtype) -> torch.Tensor:
        """A new tensor of t's shape (half a microsecond less than by shape and device)."""
        if self.stream is None:
            return torch.empty_like(t, dtype=dtype)
        with torch.cuda.stream(self.stream):
            return torch.empty_like(t, dtype=dtype)

    def empty(self, shape, dtype) -> torch.Tensor:
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.where)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.where)

    def scratch(self, nbytes: int) -> torch.Tensor:
        return self.empty((nbytes,), torch.uint8)

    def on(self) -> int:
        return _raw_stream(self.device) if self.stream is None else self.stream.cuda_stream


def _tensor(t, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    return t


# Sizes from this on are refused here: ctypes passes the low bits of a number that a C int does not hold without a word.
# (Compared where they come up: a call of about 10 us has no fraction of one for a function around it.)
_INT = 2 ** 31


def _too_large(n: int, name: str) -> ValueError:
    return ValueError(f"{name} must be below 2^31, got {n}")


def _out_dtype(dtype: Optional[torch.dtype], default: torch.dtype) -> torch.dtype:
    if dtype is None:
        return default
    if dtype not in _DT:
        raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
    return dtype


def _rows(t: torch.Tensor, name: str) -> Tuple[int, int]:
    if _tensor(t, name).dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    d = t.shape[-1]
    if d >= _INT:
        raise _too_large(d, f"the last dimension of {name}")
    return (t.numel() // d if d else 0), d


def _params_dtype(*params) -> torch.dtype:
    """The one dtype of a call's parameters (those that are None say nothing)."""
    dt = None
    for name, p in params:
        if p is None:
            continue
        if dt is not None and _tensor(p, name).dtype != dt:
            raise ValueError("the gains and a gate per channel must have one dtype")
        dt = _tensor(p, name).dtype
    if dt is not None and dt not in _DT:
        raise ValueError(f"the gains and a gate per channel must be float32 or bfloat16, got {dt}")
    return dt or torch.float32


def _gate_kind(gate, y: torch.Tensor, d: int) -> int:
    if gate is None:
        return GATE_NONE
    if y.dim() < 2:
        raise ValueError("with a gate, h and y need a row dimension")
    if _tensor(gate, "gate").shape == (d,):
        return GATE_CHANNEL
    if gate.shape == y.shape:
        return GATE_TOKEN
    raise ValueError(f"gate must have shape ({d},) or that of y, got {tuple(gate.shape)}")


@lru_cache(maxsize=1024)  # sizes alone decide it
def _norm_ws(rows: int, d: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().ttt_norm_ws_bytes(rows, d, ctypes.byref(n)), "ttt_norm_ws_bytes")
    return n.value


def ttt_norm_pre(h: torch.Tensor, w: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 x: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """The norm before a block: x = w * h * rms(h) over the last dimension (w None: no gain).

    h [...][d] float32 or bfloat16; x has h's shape and `dtype` (default: h's; a float32 h may give a bfloat16 x).
    """
    rows, d = _rows(h, "h")
    c = _Call(h.device, stream)
    ph, pw = c.arg(h, "h"), c.arg(w, "w", None, (d,))
    wdt = _params_dtype(("w", w))
    if x is None:
        x = c.like(h, _out_dtype(dtype, h.dtype))
        px = x.data_ptr()
    else:
        px = c.arg(x, "x", dtype, h.shape)
    _check(lib().ttt_norm_pre(ph, _DT[h.dtype], pw, _DT[wdt], float(eps), rows, d, px, _DT[x.dtype], c.on()),
           "ttt_norm_pre")
    return x


def ttt_norm_post(h: torch.Tensor, y: torch.Tensor, w: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
                  w_next: Optional[torch.Tensor] = None, next_norm: bool = False, o: Optional[torch.Tensor] = None,
                  x: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """After a block: o = alpha * h + beta * gate * w * y * rms(y), and with next_norm (or w_next or x given) also the
    next block's input x = w_next * o * rms(o). Returns (o, x or None).

    h [...][d] the residual stream, y (the same shape) what the block gave; gate [d], y's shape (in y's dtype) or None;
    x in `dtype` (default: y's). o may be h: the stream is then updated in place.
    """
    rows, d = _rows(h, "h")
    c = _Call(h.device, stream)
    ph, py = c.arg(h, "h"), c.arg(y, "y", None, h.shape)
    kind = _gate_kind(gate, y, d)
    pw, pn = c.arg(w, "w", None, (d,)), c.arg(w_next, "w_next", None, (d,))
    pg = c.arg(gate, "gate", y.dtype if kind == GATE_TOKEN else None)
    wdt = _params_dtype(("w", w), ("w_next", w_next), ("gate", gate if kind == GATE_CHANNEL else None))
    if o is None:
        o = c.like(h, h.dtype)
        po = o.data_ptr()
    else:
        po = c.arg(o, "o", h.dtype, h.shape)
    if x is None and (next_norm or w_next is not None):
        x = c.like(h, _out_dtype(dtype, y.dtype))
        px = x.data_ptr()
    else:
        px = c.arg(x, "x", dtype, h.shape)
    _check(lib().ttt_norm_post(ph, _DT[h.dtype], py, _DT[y.dtype], pw, pg, kind, pn, _DT[wdt], float(alpha),
                               float(beta), float(eps), rows, d, po, px, _DT[y.dtype if x is None else x.dtype],
                               c.on()), "ttt_norm_post")
    return o, x


def ttt_norm_pre_grad(dx: torch.Tensor, h: torch.Tensor, w: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      dh_in: Optional[torch.Tensor] = None, dh: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradients of ttt_norm_pre: (dh, dw) from dx; dh_in, the gradient h has from elsewhere, is added to dh (which may
    be the same tensor). dw [d] is float32, None without a gain."""
    rows, d = _rows(h, "h")
    c = _Call(h.device, stream)
    ph, pdx = c.arg(h, "h"), c.arg(dx, "dx", None, h.shape)
    pw, pin = c.arg(w, "w", None, (d,)), c.arg(dh_in, "dh_in", h.dtype, h.shape)
    wdt = _params_dtype(("w", w))
    if dh is None:
        dh = c.like(h, h.dtype)
        pdh = dh.data_ptr()
    else:
        pdh = c.arg(dh, "dh", h.dtype, h.shape)
    dw = ws = None
    nws = 0
    if w is not None:
        dw = c.empty((d,), torch.float32)
        nws = _norm_ws(rows, d)
        ws = c.scratch(nws)
    _check(lib().ttt_norm_pre_grad(pdx, _DT[dx.dtype], ph, _DT[h.dtype], pw, _DT[wdt], pin, float(eps), rows, d, pdh,
                                   dw.data_ptr() if dw is not None else None, ws.data_ptr() if ws is not None else None,
                                   nws, c.on()), "ttt_norm_pre_grad")
    return dh, dw


class NormGrads(NamedTuple):
    """What ttt_norm_post_grad gives; None where there is no such input."""

    dh: torch.Tensor
    dy: torch.Tensor
    dw: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dw_next: Optional[torch.Tensor]


def ttt_norm_post_grad(dh_in: Optional[torch.Tensor], dx: Optional[torch.Tensor], o: Optional[torch.Tensor],
                       y: torch.Tensor, w: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                       alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
                       w_next: Optional[torch.Tensor] = None, dh: Optional[torch.Tensor] = None,
                       dy: Optional[torch.Tensor] = None, stream=None) -> NormGrads:
    """Gradients of ttt_norm_post from dh_in (the gradient o has from elsewhere, or None) and dx (the gradient of x, or
    None; one of the two is needed), with o as ttt_norm_post gave it (needed with dx) and y. dh has the residual
    stream's dtype and may be dh_in; dy may be y. dw, dw_next and a [d] gate's gradient are float32."""
    rows, d = _rows(y, "y")
    c = _Call(y.device, stream)
    if dh_in is None and dx is None:
        raise ValueError("dh_in or dx must be given")
    if dx is not None and o is None:
        raise ValueError("o must be given with dx")
    hdt = _tensor(dh_in, "dh_in").dtype if dh_in is not None else _tensor(o, "o").dtype
    py, pin = c.arg(y, "y"), c.arg(dh_in, "dh_in", None, y.shape)
    pdx, po = c.arg(dx, "dx", None, y.shape), c.arg(o if dx is not None else None, "o", hdt, y.shape)
    if hdt not in _DT:
        raise ValueError(f"o must be float32 or bfloat16, got {hdt}")
    kind = _gate_kind(gate, y, d)
    pw, pn = c.arg(w, "w", None, (d,)), c.arg(w_next, "w_next", None, (d,))
    pg = c.arg(gate, "gate", y.dtype if kind == GATE_TOKEN else None)
    wdt = _params_dtype(("w", w), ("w_next", w_next), ("gate", gate if kind == GATE_CHANNEL else None))
    if dh is None:
        dh = c.like(y, hdt)
        pdh = dh.data_ptr()
    else:
        pdh = c.arg(dh, "dh", hdt, y.shape)
    if dy is None:
        dy = c.like(y, y.dtype)
        pdy = dy.data_ptr()
    else:
        pdy = c.arg(dy, "dy", y.dtype, y.shape)
    dw = c.empty((d,), torch.float32) if w is not None else None
    dn = c.empty((d,), torch.float32) if w_next is not None and dx is not None else None
    dg = None
    if kind == GATE_CHANNEL:
        dg = c.empty((d,), torch.float32)
    elif kind == GATE_TOKEN:
        dg = c.like(y, y.dtype)
    ws, nws = None, 0
    if dw is not None or dn is not None or kind == GATE_CHANNEL:
        nws = _norm_ws(rows, d)
        ws = c.scratch(nws)
    out = [None if t is None else t.data_ptr() for t in (dw, dg, dn, ws)]
    _check(lib().ttt_norm_post_grad(pin, pdx, _DT[y.dtype if dx is None else dx.dtype], po, _DT[hdt], py, _DT[y.dtype],
                                    pw, pg, kind, pn, _DT[wdt], float(alpha), float(beta), float(eps), rows, d, pdh,
                                    pdy, out[0], out[1], out[2], out[3], nws, c.on()), "ttt_norm_post_grad")
    return NormGrads(dh, dy, dw, dg, dn)


def _ids_arg(c: _Call, ids: torch.Tensor) -> Tuple[int, int, int, int]:
    """(address, row stride, rows, tokens per row) of a call's ids: int32, contiguous, or 2-D with rows apart (a
    [:, :T] view of the layer's [B][T+1] ids)."""
    if _tensor(ids, "ids").dtype != torch.int32:
        raise ValueError(f"ids must be {torch.int32}, got {ids.dtype}")
    n = ids.numel()
    if n >= _INT:
        raise _too_large(n, "the number of ids")
    if not ids.is_cuda:
        raise ValueError("ids must be a device tensor")
    if ids.get_device() != c.device:
        raise ValueError("ids must be on the current device")
    if c.stream is not None:
        ids.record_stream(c.stream)
    if ids.dim() == 2 and not ids.is_contiguous():
        B, T = ids.shape
        if ids.stride(1) != 1 or ids.stride(0) < T:
            raise ValueError("ids must be contiguous or a 2-D view of contiguous rows")
        return ids.data_ptr(), ids.stride(0), B, T
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous or a 2-D view of contiguous rows")
    return ids.data_ptr(), n, 1, n


@lru_cache(maxsize=1024)
def _embed_ws(B: int, T: int, vocab: int, d: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().ttt_embed_grad_ws_bytes(B, T, vocab, d, ctypes.byref(n)), "ttt_embed_grad_ws_bytes")
    return n.value


@lru_cache(maxsize=1024)
def _grad_ws(n: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().ttt_grad_ws_bytes(n, ctypes.byref(b)), "ttt_grad_ws_bytes")
    return b.value


def ttt_embed(E: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, x: Optional[torch.Tensor] = None,
              dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """Token embedding: x[t] = scale * E[ids[t]], a zero row for an id outside [0, vocab).

    E [vocab][d]; ids int32 of any shape, or a 2-D view of contiguous rows; x is ids.shape + (d,) in `dtype` (default:
    the table's)."""
    if _tensor(E, "E").dim() != 2:
        raise ValueError("E must be [vocab][d]")
    vocab, d = E.shape
    if vocab >= _INT or d >= _INT:
        raise _too_large(max(vocab, d), "each dimension of E")
    c = _Call(E.device, stream)
    pE = c.arg(E, "E")
    pi, ld, B, T = _ids_arg(c, ids)
    shape = ids.shape + (d,)
    if x is None:
        x = c.empty(shape, _out_dtype(dtype, E.dtype))
        px = x.data_ptr()
    else:
        px = c.arg(x, "x", dtype, shape)
    _check(lib().ttt_embed(pE, _DT[E.dtype], vocab, d, pi, ld, B, T, float(scale), px, _DT[x.dtype], c.on()),
           "ttt_embed")
    return x


def ttt_embed_grad(dx: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0,
                   dE: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32, accumulate: bool = False,
                   stream=None) -> torch.Tensor:
    """Gradient of ttt_embed's table: dE[v] = scale * sum of dx[t] over ids[t] = v, [vocab][d] in `dtype` (or that of
    a given dE). With accumulate the sums are added to dE, which must then be given."""
    c = _Call(_tensor(dx, "dx").device, stream)
    vocab, d = int(vocab), dx.shape[-1] if dx.dim() else 0
    if not -_INT < vocab < _INT:
        raise _too_large(vocab, "vocab")
    if d >= _INT:
        raise _too_large(d, "the last dimension of dx")
    pi, ld, B, T = _ids_arg(c, ids)
    if dx.dim() != ids.dim() + 1 or dx.shape[:-1] != ids.shape:
        raise ValueError(f"dx must be ids' shape and d, got {tuple(dx.shape)} for ids {tuple(ids.shape)}")
    pdx = c.arg(dx, "dx")
    if dE is None:
        if accumulate:
            raise ValueError("dE must be given to accumulate into")
        dE = c.empty((vocab, d), _out_dtype(dtype, torch.float32))
        pE = dE.data_ptr()
    else:
        pE = c.arg(dE, "dE", None, (vocab, d))
    nws = _embed_ws(B, T, vocab, d)
    ws = c.scratch(nws)
    _check(lib().ttt_embed_grad(pdx, _DT[dx.dtype], pi, ld, B, T, float(scale), vocab, d, pE, _DT[dE.dtype],
                                1 if accumulate else 0, ws.data_ptr(), nws, c.on()), "ttt_embed_grad")
    return dE


class _Many:
    """Lists of tensors as the library takes them: host arrays of addresses, element counts and types. The attributes
    are read by map() over the methods themselves: at hundreds of tensors this loop is what a call costs. A list entry
    that is no tensor ends in their TypeError."""

    _dtype = staticmethod(attrgetter("dtype"))

    def __init__(self, c: _Call, grads):
        self.n = len(grads)
        self.sizes = array("q", map(torch.Tensor.numel, grads))
        self.dtypes = list(map(self._dtype, grads))
        found = set(self.dtypes)
        if not _DT.keys() >= found:
            raise ValueError("grads must be float32 or bfloat16")
        if len(found) == 1:
            kinds = array("i", [_DT[found.pop()]]) * self.n
        else:
            kinds = array("i", map(_DT.__getitem__, self.dtypes))
        self._keep = (self._addresses(c, grads, "grads"), self.sizes, kinds)
        self.args = tuple(a.buffer_info()[0] for a in self._keep) + (self.n,)

    @staticmethod
    def _addresses(c: _Call, ts, name: str) -> array:
        if not all(map(torch.Tensor.is_contiguous, ts)):
            raise ValueError(f"{name} must be contiguous")
        where = set(map(torch.Tensor.get_device, ts))  # -1 for host tensors
        if -1 in where:
            raise ValueError(f"{name} must be device tensors")
        if not where <= {c.device}:
            raise ValueError(f"{name} must be on the current device")
        if c.stream is not None:
            for t in ts:
                t.record_stream(c.stream)
        return array("Q", map(torch.Tensor.data_ptr, ts))

    def outputs(self, c: _Call, out) -> array:
        if len(out) != self.n:
            raise ValueError(f"out must have one tensor per gradient, got {len(out)} for {self.n}")
        if array("q", map(torch.Tensor.numel, out)) != self.sizes or list(map(self._dtype, out)) != self.dtypes:
            raise ValueError("out must have the gradients' dtypes and sizes")
        return self._addresses(c, out, "out")


def _grads_call(grads, norm, stream):
    grads = list(grads)
    where = grads[0].device if grads and isinstance(grads[0], torch.Tensor) else torch.device("cuda")
    c = _Call(where, stream)
    m = _Many(c, grads)
    if norm is None:
        norm = c.empty((1,), torch.float32)
        pn = norm.data_ptr()
    else:
        pn = c.arg(norm, "norm", torch.float32, (1,))
    nws = _grad_ws(m.n)
    return c, m, norm, pn, c.scratch(nws), nws


def ttt_grad_norm(grads, norm: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The 2-norm of all the tensors together, as a float32 device tensor of one element. grads: a list of contiguous
    float32 or bfloat16 tensors."""
    c, m, norm, pn, ws, nws = _grads_call(grads, norm, stream)
    _check(lib().ttt_grad_norm(*m.args, pn, ws.data_ptr(), nws, c.on()), "ttt_grad_norm")
    return norm


def ttt_clip_grads(grads, tau: float, out=None, norm: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scales the gradients by min(1, tau / N), N the 2-norm of them all, in place or into `out` (a list of tensors like
    them). Returns N as it was before, a float32 device tensor of one element. Where N is not finite the gradients
    stay as they are."""
    c, m, norm, pn, ws, nws = _grads_call(grads, norm, stream)
    po = None if out is None else m.outputs(c, out)
    _check(lib().ttt_clip_grads(*m.args, float(tau), None if po is None else po.buffer_info()[0], pn, ws.data_ptr(),
                                nws, c.on()), "ttt_clip_grads")
    return norm

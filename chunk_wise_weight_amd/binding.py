"""Python binding of libttt.so: the C ABI's entry points under the same names.

Argument marshalling only: tensors are turned into device pointers and sizes,
and torch's current HIP stream is passed along. Every step of the
computation runs in the library's HIP kernels; there is no fallback path, and
a missing or unloadable library raises.
"""
from __future__ import annotations

import ctypes
import os
import sys
import warnings
from array import array
from functools import lru_cache
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
           "ttt_clip_grads", "ttt_linear_ws_bytes", "ttt_linear", "ttt_gated_ws_bytes", "ttt_gated",
           "ttt_linear_grad_ws_bytes", "ttt_linear_grad", "ttt_gated_grad_ws_bytes", "ttt_gated_grad",
           "ttt_dense_plan", "ttt_adamw", "ttt_adamw_values")

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
    psz, f64 = ctypes.POINTER(sz), ctypes.c_double
    for fn in (L.ttt_linear_ws_bytes, L.ttt_gated_ws_bytes, L.ttt_gated_grad_ws_bytes):
        fn.argtypes = [i64, i32, i32, i32, psz]
        fn.restype = i32
    L.ttt_linear_grad_ws_bytes.argtypes = [i64, i32, i32, i32, i32, i32, psz]
    L.ttt_linear_grad_ws_bytes.restype = i32
    L.ttt_linear.argtypes = [vp, vp, i32, vp, i32, f32, vp, i64, i32, i32, vp, vp, i32, vp, sz, vp]
    L.ttt_gated.argtypes = [vp, vp, vp, i32, vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, sz, vp]
    L.ttt_linear_grad.argtypes = [vp, i32, vp, vp, i32, vp, i32, f32, i64, i32, i32, vp, vp, vp, i32, vp, sz, vp]
    L.ttt_gated_grad.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    L.ttt_dense_plan.argtypes = [i32, i64, i32, i32, i32, i32, ip, ip, ip, ip]
    L.ttt_dense_plan.restype = i32
    L.ttt_adamw.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, i32, i64, vp, f64, vp, f64, f64, f64, f64, vp,
                            f64, ctypes.c_uint32, vp]
    L.ttt_adamw_values.argtypes = [vp, vp, i32, vp, vp, i32, vp]
    for fn in (L.ttt_linear, L.ttt_gated, L.ttt_linear_grad, L.ttt_gated_grad, L.ttt_adamw, L.ttt_adamw_values):
        fn.restype = i32
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


_KINDS = {torch.float32: TTT_F32, torch.bfloat16: TTT_BF16, torch.uint8: 2, torch.int16: 3}


def _read_python(ts: list, name: str, device: int):
    """What the native reader (csrc/tensor_lists.cpp) gives, for where it is not there: half a microsecond a tensor (a
    step over 144 tensors, 720 in its lists, 375 us; 18 with the native one)."""
    at, numel, kinds, seen, faults = array("Q"), array("q"), array("i"), 0, 0
    for t in ts:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be tensors, got {type(t).__name__}")
        fault = (1 if t.layout != torch.strided or not t.is_contiguous() else 2 if not t.is_cuda else
                 4 if t.get_device() != device else 0)
        kind = _KINDS.get(t.dtype, 4)
        at.append(0 if fault else t.data_ptr())
        numel.append(t.numel())
        kinds.append(kind)
        seen |= 1 << kind
        faults |= fault
    return at.tobytes(), numel.tobytes(), kinds.tobytes(), seen, faults


def built_for() -> str:
    """The torch and Python that a native reader must have been built for."""
    return f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


_read = None


def _reader():
    """The reader of tensor lists (chosen once): native, or in Python where no native one was built for this torch and
    Python."""
    global _read
    if _read is None:
        try:
            from . import _tensor_lists
            other = getattr(_tensor_lists, "built_for", "another torch")
            if other != built_for():
                raise ImportError(f"it was built for {other}, this is {built_for()}")
            _read = _tensor_lists.read
        except ImportError as e:
            warnings.warn(f"lists of tensors are read in Python, half a microsecond a tensor: no _tensor_lists.so ({e}); "
                          "run `python -m chunk_wise_weight_amd.build`", RuntimeWarning, stacklevel=2)
            _read = _read_python
    return _read


class _Read:
    """Addresses, element counts and types of a list of tensors, each as the bytes of an array that the library reads
    during the call."""

    __slots__ = ("at", "numel", "kinds", "seen", "n")

    def __init__(self, c: _Call, ts: list, name: str, types: int, what: str):
        """types: a mask of those allowed, 1 << type (TTT_F32, TTT_BF16, 2 for uint8, 3 for int16); what: their names."""
        self.at, self.numel, self.kinds, self.seen, faults = _reader()(ts, name, c.device)
        self.n = len(ts)
        if self.seen & ~types:
            raise ValueError(f"{name} must be {what}")
        if faults:
            raise ValueError(f"{name} must be " + ("contiguous" if faults & 1 else "device tensors" if faults & 2 else
                                                   "on the current device"))
        if c.stream is not None:
            for t in ts:
                t.record_stream(c.stream)


_FLOATS = (1 << TTT_F32 | 1 << TTT_BF16, "float32 or bfloat16")


class _Many:
    """Lists of tensors as the library takes them: host arrays of addresses, element counts and types."""

    def __init__(self, c: _Call, grads):
        self.read = r = _Read(c, grads, "grads", *_FLOATS)
        self.args = (r.at, r.numel, r.kinds, r.n)

    def outputs(self, c: _Call, out) -> bytes:
        out = list(out)
        if len(out) != self.read.n:
            raise ValueError(f"out must have one tensor per gradient, got {len(out)} for {self.read.n}")
        r = _Read(c, out, "out", *_FLOATS)
        if r.numel != self.read.numel or r.kinds != self.read.kinds:
            raise ValueError("out must have the gradients' dtypes and sizes")
        return r.at


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
    nws = _grad_ws(m.read.n)
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
    _check(lib().ttt_clip_grads(*m.args, float(tau), po, pn, ws.data_ptr(),
                                nws, c.on()), "ttt_clip_grads")
    return norm


# ---- the plain layers and the step ----

_ACT = {None: 0, "silu": 1, "gelu": 2, "relu": 3}  # TTT_ACT_* in include/ttt.h


def _act(act: Optional[str], gated: bool = False) -> int:
    if act not in _ACT or (gated and act is None):
        names = [a for a in _ACT if a is not None or not gated]
        raise ValueError(f"act must be one of {names}, got {act!r}")
    return _ACT[act]


@lru_cache(maxsize=1024)
def _dense_ws(name: str, rows: int, n_in: int, n_out: int, dt: int, *more: int) -> int:
    n = ctypes.c_size_t()
    _check(getattr(lib(), name)(rows, n_in, n_out, dt, *more, ctypes.byref(n)), name)
    return n.value


def _weight_shape(w: torch.Tensor, name: str, n_in: int) -> int:
    """The rows of a weight [out][in]."""
    if _tensor(w, name).dim() != 2 or w.shape[1] != n_in:
        raise ValueError(f"{name} must be [out][{n_in}], got {tuple(w.shape)}")
    if w.shape[0] >= _INT:
        raise _too_large(w.shape[0], f"the first dimension of {name}")
    return w.shape[0]


def ttt_linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, act: Optional[str] = None,
               residual: Optional[torch.Tensor] = None, scale: float = 1.0, keep: bool = False,
               y: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None, stream=None):
    """y = residual + scale * act(x w^T + bias); act None, "silu", "gelu" (tanh form) or "relu".

    x [...][in], w [out][in], bias [out], all of one dtype; y [...][out] in `dtype` (default: the residual's, else x's;
    a bfloat16 x may give a float32 y), the residual in y's dtype. y may be the residual. With keep returns (y, pre),
    pre = x w^T + bias in x's dtype, which ttt_linear_grad takes where there is an activation."""
    rows, n = _rows(x, "x")
    out = _weight_shape(w, "w", n)
    c = _Call(x.device, stream)
    dt = x.dtype
    px, pw, pb = c.arg(x, "x"), c.arg(w, "w", dt), c.arg(bias, "bias", dt, (out,))
    shape = x.shape[:-1] + (out,)
    if y is None:
        y = c.empty(shape, _out_dtype(dtype, dt if residual is None else _tensor(residual, "residual").dtype))
        py = y.data_ptr()
    else:
        py = c.arg(y, "y", dtype, shape)
    pr = c.arg(residual, "residual", y.dtype, shape)
    pre = c.empty(shape, dt) if keep else None
    nws = _dense_ws("ttt_linear_ws_bytes", rows, n, out, _DT[dt])
    ws = c.scratch(nws) if nws else None
    _check(lib().ttt_linear(px, pw, _DT[dt], pb, _act(act), float(scale), pr, rows, n, out,
                            None if pre is None else pre.data_ptr(), py, _DT[y.dtype],
                            None if ws is None else ws.data_ptr(), nws, c.on()), "ttt_linear")
    return (y, pre) if keep else y


def ttt_gated(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, b_gate: Optional[torch.Tensor] = None,
              b_up: Optional[torch.Tensor] = None, act: str = "silu", keep: bool = False,
              z: Optional[torch.Tensor] = None, stream=None):
    """The gated projections of a feed-forward block: z = act(g) * u, g = x w_gate^T + b_gate, u = x w_up^T + b_up.

    x [...][in], weights [f][in], biases [f] (both or neither), z [...][f], all of one dtype; act "silu", "gelu" (tanh
    form) or "relu". With keep returns (z, g, u) for ttt_gated_grad."""
    rows, n = _rows(x, "x")
    f = _weight_shape(w_gate, "w_gate", n)
    c = _Call(x.device, stream)
    dt = x.dtype
    px, pg, pu = c.arg(x, "x"), c.arg(w_gate, "w_gate", dt), c.arg(_tensor(w_up, "w_up"), "w_up", dt, (f, n))
    pbg, pbu = c.arg(b_gate, "b_gate", dt, (f,)), c.arg(b_up, "b_up", dt, (f,))
    shape = x.shape[:-1] + (f,)
    if z is None:
        z = c.empty(shape, dt)
        pz = z.data_ptr()
    else:
        pz = c.arg(z, "z", dt, shape)
    g, u = (c.empty(shape, dt), c.empty(shape, dt)) if keep else (None, None)
    nws = _dense_ws("ttt_gated_ws_bytes", rows, n, f, _DT[dt])
    ws = c.scratch(nws) if nws else None
    _check(lib().ttt_gated(px, pg, pu, _DT[dt], pbg, pbu, _act(act, True), rows, n, f,
                           None if g is None else g.data_ptr(), None if u is None else u.data_ptr(), pz,
                           None if ws is None else ws.data_ptr(), nws, c.on()), "ttt_gated")
    return (z, g, u) if keep else z


class LinearGrads(NamedTuple):
    """What ttt_linear_grad gives; None where it was not asked for."""

    dx: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


class GatedGrads(NamedTuple):
    """What ttt_gated_grad gives; None where it was not asked for."""

    dx: Optional[torch.Tensor]
    dw_gate: Optional[torch.Tensor]
    dw_up: Optional[torch.Tensor]
    db_gate: Optional[torch.Tensor]
    db_up: Optional[torch.Tensor]


def _grad_out(c: _Call, given, name: str, wanted: bool, accumulate: bool, shape, dtype):
    """(tensor, address) of a gradient: given, made here, or not wanted."""
    if given is not None:
        return given, c.arg(given, name, dtype, shape)
    if not wanted:
        return None, None
    if accumulate:
        raise ValueError(f"{name} must be given to accumulate into")
    t = c.empty(shape, dtype)
    return t, t.data_ptr()


def ttt_linear_grad(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, act: Optional[str] = None,
                    pre: Optional[torch.Tensor] = None, scale: float = 1.0, bias: bool = False,
                    dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                    dbias: Optional[torch.Tensor] = None, need_dx: bool = True, need_dw: bool = True,
                    accumulate: bool = False, stream=None) -> LinearGrads:
    """Gradients of ttt_linear: with q = scale * dy * act'(pre), dx = q w, dw = q^T x and, with bias, dbias = sum q.

    dy [...][out] in the dtype y had; pre as ttt_linear kept it (needed with an activation). dx and dw have x's dtype,
    dbias is float32. With a bfloat16 x the products take q rounded to bfloat16, also from a float32 dy; with float32 x
    and w nothing is rounded to fewer bits. With accumulate, dw and dbias are added to the tensors given for them."""
    rows, n = _rows(x, "x")
    out = _weight_shape(w, "w", n)
    c = _Call(x.device, stream)
    dt, kind = x.dtype, _act(act)
    px, pw = c.arg(x, "x"), c.arg(w, "w", dt)
    shape = x.shape[:-1] + (out,)
    pdy = c.arg(_tensor(dy, "dy"), "dy", None, shape)
    if kind and pre is None:
        raise ValueError("pre must be given with an activation")
    pp = c.arg(pre if kind else None, "pre", dt, shape)
    dx, pdx = _grad_out(c, dx, "dx", need_dx, False, x.shape, dt)
    dw, pdw = _grad_out(c, dw, "dw", need_dw, accumulate, (out, n), dt)
    dbias, pdb = _grad_out(c, dbias, "dbias", bias, accumulate, (out,), torch.float32)
    nws = _dense_ws("ttt_linear_grad_ws_bytes", rows, n, out, _DT[dt], _DT[dy.dtype], kind)
    ws = c.scratch(nws)
    _check(lib().ttt_linear_grad(pdy, _DT[dy.dtype], px, pw, _DT[dt], pp, kind, float(scale), rows, n, out, pdx, pdw,
                                 pdb, 1 if accumulate else 0, ws.data_ptr(), nws, c.on()), "ttt_linear_grad")
    return LinearGrads(dx, dw, dbias)


def ttt_gated_grad(dz: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, g: torch.Tensor,
                   u: torch.Tensor, act: str = "silu", bias: bool = False, dx: Optional[torch.Tensor] = None,
                   dw_gate: Optional[torch.Tensor] = None, dw_up: Optional[torch.Tensor] = None,
                   db_gate: Optional[torch.Tensor] = None, db_up: Optional[torch.Tensor] = None, need_dx: bool = True,
                   need_dw: bool = True, accumulate: bool = False, stream=None) -> GatedGrads:
    """Gradients of ttt_gated: with dg = dz * u * act'(g) and du = dz * act(g), dx = dg w_gate + du w_up,
    dw_gate = dg^T x, dw_up = du^T x and, with bias, db_gate = sum dg, db_up = sum du.

    g, u as ttt_gated kept them. dx and the weights' gradients have x's dtype, the biases' are float32; the products
    take dg and du rounded to x's dtype. With accumulate the weights' and biases' gradients are added to the tensors
    given for them."""
    rows, n = _rows(x, "x")
    f = _weight_shape(w_gate, "w_gate", n)
    c = _Call(x.device, stream)
    dt, kind = x.dtype, _act(act, True)
    px, pg, pu = c.arg(x, "x"), c.arg(w_gate, "w_gate", dt), c.arg(_tensor(w_up, "w_up"), "w_up", dt, (f, n))
    shape = x.shape[:-1] + (f,)
    pdz = c.arg(_tensor(dz, "dz"), "dz", dt, shape)
    pkg, pku = c.arg(_tensor(g, "g"), "g", dt, shape), c.arg(_tensor(u, "u"), "u", dt, shape)
    dx, pdx = _grad_out(c, dx, "dx", need_dx, False, x.shape, dt)
    dw_gate, pdg = _grad_out(c, dw_gate, "dw_gate", need_dw, accumulate, (f, n), dt)
    dw_up, pdu = _grad_out(c, dw_up, "dw_up", need_dw, accumulate, (f, n), dt)
    db_gate, pbg = _grad_out(c, db_gate, "db_gate", bias, accumulate, (f,), torch.float32)
    db_up, pbu = _grad_out(c, db_up, "db_up", bias, accumulate, (f,), torch.float32)
    nws = _dense_ws("ttt_gated_grad_ws_bytes", rows, n, f, _DT[dt])
    ws = c.scratch(nws)
    _check(lib().ttt_gated_grad(pdz, px, pg, pu, _DT[dt], pkg, pku, kind, rows, n, f, pdx, pdg, pdu, pbg, pbu,
                                1 if accumulate else 0, ws.data_ptr(), nws, c.on()), "ttt_gated_grad")
    return GatedGrads(dx, dw_gate, dw_up, db_gate, db_up)


_PRODUCTS = ("linear", "gated", "linear_dx", "linear_dw", "gated_dx", "gated_dw")  # TTT_PRODUCT_* in include/ttt.h
_KERNELS = ("few", "direct", "general")  # TTT_KERNEL_*


def ttt_dense_plan(product: str, rows: int, n_in: int, n_out: int, dtype: torch.dtype, q_made: bool = False) -> Dict:
    """How a product of ttt_linear, ttt_gated or their gradients runs on arrays that start on 16 bytes, as a dict of
    kernel ("few", "direct" or "general"), tile, splits and copies; host-only, works without a GPU. product: "linear",
    "gated", "linear_dx", "linear_dw", "gated_dx" or "gated_dw". q_made: ttt_linear_grad has an activation, or dy
    another dtype than x."""
    if product not in _PRODUCTS:
        raise ValueError(f"product must be one of {list(_PRODUCTS)}, got {product!r}")
    if dtype not in _DT:
        raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
    for n, name in ((n_in, "n_in"), (n_out, "n_out")):
        if n >= _INT:
            raise _too_large(n, name)
    got = [ctypes.c_int() for _ in range(4)]
    _check(lib().ttt_dense_plan(_PRODUCTS.index(product), rows, n_in, n_out, _DT[dtype],
                                1 if q_made else 0, *map(ctypes.byref, got)), "ttt_dense_plan")
    kernel, tile, splits, copies = (v.value for v in got)
    return {"kernel": _KERNELS[kernel], "tile": tile, "splits": splits, "copies": copies}


_F32_ONLY, _BF16_ONLY = (1 << TTT_F32, "torch.float32"), (1 << TTT_BF16, "torch.bfloat16")
_CODES, _TOPS = (1 << 2, "torch.uint8"), (1 << 3, "torch.int16")


def _sized(c: _Call, ts, name: str, types, like: _Read) -> _Read:
    """A list with a tensor of each parameter's size."""
    ts = list(ts)
    if len(ts) != like.n:
        raise ValueError(f"{name} must have one tensor per parameter, got {len(ts)} for {like.n}")
    r = _Read(c, ts, name, *types)
    if r.numel != like.numel:
        raise ValueError(f"{name} must have the parameters' sizes")
    return r


def _tops(c: _Call, ts, like: _Read) -> _Read:
    ts = list(ts)
    r = _Read(c, ts, "tops", *_TOPS)
    if [tuple(t.shape) for t in ts] != [(2, -(-n // 256)) for n in array("q", like.numel)]:
        raise ValueError("tops must have one tensor [2][ceil(numel / 256)] per parameter")
    return r


def _list_call(ts, stream) -> _Call:
    return _Call(ts[0].device if ts and isinstance(ts[0], torch.Tensor) else torch.device("cuda"), stream)


def _number(c: _Call, v, name: str, dtype) -> Tuple[object, Optional[int]]:
    """A number, or a device tensor of one element: (the number, the tensor's address)."""
    if not isinstance(v, torch.Tensor):
        return v, None
    if v.dtype != dtype or v.numel() != 1:
        raise ValueError(f"{name} must be a number or a {dtype} tensor of one element")
    if v.get_device() != c.device or c.device < 0:
        raise ValueError(f"{name} must be {'on the current device' if v.is_cuda else 'a number or a device tensor'}")
    if c.stream is not None:
        v.record_stream(c.stream)
    return 0, v.data_ptr()


def ttt_adamw(params, grads, m, v, step, lr, betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
              weight_decay: float = 0.01, copies=None, norm: Optional[torch.Tensor] = None, tau: float = float("inf"),
              tops=None, seed: int = 0, stream=None) -> None:
    """One AdamW step over lists of contiguous tensors, in place:

        g' = g min(1, tau / norm);  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
        w = w (1 - lr weight_decay) - lr (m / (1 - b1^step)) / (sqrt(v / (1 - b2^step)) + eps)

    params and grads are float32 or bfloat16, each tensor its own. The moments m and v are float32, or uint8 codes with
    `tops`, int16 [2][ceil(numel / 256)] per parameter (all zeros at the start, as the codes): see include/ttt.h for
    what a code stands for, ttt_adamw_values for its values. They are rounded at random, by `seed`, the step and the
    place. copies: bfloat16 tensors that receive the rounded parameters. norm: what ttt_grad_norm gave for the
    gradients; one that is not finite clips nothing, and without one tau does not count. step (1, 2, ...) and lr are
    numbers, or device tensors of one element (int64, float32) that a captured call reads anew at each replay."""
    params, m = list(params), list(m)
    bits8 = bool(m) and _tensor(m[0], "m").dtype == torch.uint8
    if bits8 and tops is None:
        raise ValueError("tops must be given with codes")
    if not 0 <= seed < 2 ** 32:
        raise ValueError(f"seed must be in [0, 2^32), got {seed}")
    c = _list_call(params, stream)
    p = _Read(c, params, "params", *_FLOATS)
    g = _sized(c, grads, "grads", _FLOATS, p)
    state = _CODES if bits8 else _F32_ONLY
    m, v = _sized(c, m, "m", state, p), _sized(c, v, "v", state, p)
    top = _tops(c, tops, p).at if bits8 else None
    cs = None if copies is None else _sized(c, copies, "copies", _BF16_ONLY, p).at
    step, step_dev = _number(c, step, "step", torch.int64)
    lr, lr_dev = _number(c, lr, "lr", torch.float32)
    if not -2 ** 63 <= step < 2 ** 63:
        raise ValueError(f"step must be below 2^63, got {step}")
    _check(lib().ttt_adamw(p.at, p.kinds, g.at, g.kinds, m.at, v.at, 8 if bits8 else 32, top, cs, p.numel, p.n,
                           int(step), step_dev, float(lr), lr_dev, float(betas[0]), float(betas[1]), float(eps),
                           float(weight_decay), c.arg(norm, "norm", torch.float32, (1,)), float(tau), int(seed),
                           c.on()), "ttt_adamw")


def ttt_adamw_values(codes, tops, moment: int, out=None, stream=None) -> List[torch.Tensor]:
    """The float32 values of ttt_adamw's 8-bit moments: moment 1 (codes m) or 2 (codes v), a tensor of each one's shape
    (or into `out`)."""
    codes = list(codes)
    c = _list_call(codes, stream)
    r = _Read(c, codes, "codes", *_CODES)
    top = _tops(c, tops, r)
    out = [c.like(t, torch.float32) for t in codes] if out is None else list(out)
    o = _sized(c, out, "out", _F32_ONLY, r)
    _check(lib().ttt_adamw_values(r.at, top.at, int(moment), o.at, r.numel, r.n, c.on()), "ttt_adamw_values")
    return out

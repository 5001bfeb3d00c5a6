"""Selective-scan forward and pscan on GB300 (sm_103a): the Python binding.

The computation lives in ``libsscan.so`` (hand-written CUDA kernels behind
the C ABI of ``include/sscan.h``).  This module only checks tensor shapes,
dtypes and devices, allocates outputs with torch, and passes raw pointers and
the current CUDA stream through ctypes.  There is no fallback: if the library
is missing or fails to load, every call raises.

    y, h_last = sscan_fwd(u, delta, A, B, C, D=None, h0=None)
    h = pscan(a, b, h0=None)

Shapes: u, delta [batch, dim, L] (float32 or bfloat16); A [dim, N] float32;
B, C [batch, N, L] (same dtype as u); D [dim] float32; h0 [batch, dim, N]
float32.  Returns y [batch, dim, L] in the I/O dtype and the final state
[batch, dim, N] float32.

The operators around the scan in a layer: ``sconv_fwd`` / ``sconv_bwd`` (short
causal convolution), ``addnorm_fwd`` / ``addnorm_bwd`` (RMS norm with the residual addition),
``gatenorm_fwd`` / ``gatenorm_bwd`` (gated RMS norm over the scan's channels); and for requests over
a cache of states ``sconv_prompt`` and ``sscan_prompt`` (packed prompts),
``sconv_step``, ``sscan_step`` and ``gatenorm_step`` (single tokens).

Linear attention with a decay for each head (the scan with one rate a head and a
matrix of states): ``lattn_fwd`` / ``lattn_bwd``, ``lattn_prompt`` and
``lattn_step``; the norms of its queries and keys for each head with the rotation by
position: ``qknorm_fwd`` / ``qknorm_bwd`` and ``qknorm_step``; and ``state_move``, which
copies, forks, compacts and frees rows of a cache of states.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from ._build import LIB as LIB_PATH

SSCAN_OK, SSCAN_ERR_INVALID, SSCAN_ERR_CUDA, SSCAN_ERR_TIMEOUT = 0, 1, 2, 3
SSCAN_F32, SSCAN_BF16 = 0, 1
SSCAN_DELTA_SOFTPLUS, SSCAN_ZOH = 1, 2
SCONV_SILU, SCONV_MAX_WIDTH = 1, 4
GATENORM_NORM_FIRST, BLOCKNORM_MAX_WIDTH = 1, 16384
LATTN_MAX_KEY, LATTN_MAX_VALUE, QKNORM_MAX_DIM, STATE_MOVE_MAX = 128, 256, 256, 8192

_vp, _fp, _i64, _int = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_f32 = ctypes.c_float
_lock = threading.Lock()
_lib = None

# name -> (restype, argtypes): every symbol include/sscan.h declares
SIGNATURES = {
    "sscan_fwd": (_int, [_vp, _vp, _fp, _vp, _vp, _fp, _fp, _vp, _fp,
                         _i64, _i64, _i64, _i64, _int, _vp]),
    "sscan_fwd_ex": (_int, [_vp, _vp, _fp, _vp, _vp, _fp, _fp, _vp, _fp,
                            _i64, _i64, _i64, _i64, _int, _int, _int, _vp]),
    "sscan_fwd_fused": (_int, [_vp, _vp, _fp, _vp, _vp, _fp, _vp, _fp, _fp, _vp, _fp,
                               _i64, _i64, _i64, _i64, _int, _int, _int, _int, _vp]),
    "sscan_fwd_noalloc": (_int, [_vp, _vp, _fp, _vp, _vp, _fp, _fp, _vp, _fp,
                                 _i64, _i64, _i64, _i64, _int, _int, _vp]),
    "sscan_bwd": (_int, [_vp, _vp, _fp, _vp, _vp, _fp, _fp, _vp, _fp, _vp, _vp, _fp, _fp, _fp, _fp,
                         _fp, _i64, _i64, _i64, _i64, _int, _vp]),
    "sscan_step": (_int, [_vp, _vp, _fp, _vp, _vp, _fp, _fp, _vp, _i64, _i64, _i64, _int, _vp]),
    "sscan_step_slots": (_int, [_vp] * 11 + [_i64] * 5 + [_int, _int, _vp]),
    "sscan_prompt": (_int, [_vp] * 13 + [_i64] * 5 + [_int, _int, _int, _vp]),
    "sconv_fwd": (_int, [_vp] * 6 + [_i64] * 6 + [_int, _int, _vp]),
    "sconv_bwd": (_int, [_vp] * 10 + [_i64] * 6 + [_int, _int, _vp]),
    "sconv_prompt": (_int, [_vp] * 8 + [_i64] * 6 + [_int, _int, _vp]),
    "sconv_step": (_int, [_vp] * 6 + [_i64] * 5 + [_int, _int, _vp]),
    "addnorm_fwd": (_int, [_vp] * 5 + [_i64] * 2 + [_f32, _f32, _int, _vp]),
    "addnorm_bwd": (_int, [_vp] * 7 + [_i64] * 2 + [_f32, _f32, _int, _vp]),
    "gatenorm_fwd": (_int, [_vp] * 4 + [_i64] * 6 + [_f32, _int, _int, _vp]),
    "gatenorm_bwd": (_int, [_vp] * 7 + [_i64] * 6 + [_f32, _int, _int, _vp]),
    "gatenorm_step": (_int, [_vp] * 4 + [_i64] * 4 + [_f32, _int, _int, _vp]),
    "lattn_fwd": (_int, [_vp] * 10 + [_i64] * 6 + [_vp, _f32, _int, _int, _int, _vp]),
    "lattn_bwd": (_int, [_vp] * 18 + [_i64] * 6 + [_vp, _f32, _int, _int, _vp]),
    "lattn_prompt": (_int, [_vp] * 12 + [_i64] * 7 + [_vp, _f32, _int, _int, _int, _vp]),
    "lattn_step": (_int, [_vp] * 10 + [_i64] * 10 + [_f32, _int, _int, _vp]),
    "qknorm_fwd": (_int, [_vp] * 8 + [_i64] * 6 + [_vp, _f32, _int, _vp]),
    "qknorm_bwd": (_int, [_vp] * 12 + [_i64] * 6 + [_vp, _f32, _int, _vp]),
    "qknorm_step": (_int, [_vp] * 8 + [_i64] * 7 + [_f32, _int, _vp]),
    "state_move": (_int, [_vp] * 3 + [_i64] * 4 + [_vp]),
    "pscan": (_int, [_fp, _fp, _fp, _fp, _i64, _i64, _vp]),
    "sscan_status_string": (ctypes.c_char_p, [_int]),
    "sscan_get_last_error": (_int, []),
    "sscan_max_dstate": (_int, []),
    "sscan_debug_expire_next_wait": (None, [ctypes.c_uint]),
    "sscan_debug_expire_next_correction_wait": (None, [ctypes.c_uint]),
    "sscan_probe_ex2": (_int, [_fp, _int, _int, _vp]),
    "sscan_probe_ex2_count": (ctypes.c_longlong, [_int, _int]),
    "sscan_probe_element": (_int, [_fp, _int, _int, _int, _vp]),
    "sscan_probe_element_count": (ctypes.c_longlong, [_int, _int, _int]),
    "sscan_last_launch_count": (_int, []),
    "sscan_last_plan": (ctypes.c_char_p, []),
}


class SscanError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load_library(path: str | None = None):
    """Load libsscan.so (building it first if this tree has sources but no
    library).  ``path``, else the SSCAN_LIBRARY environment variable, selects
    another build of the library.  Raises if it cannot be loaded."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or os.environ.get("SSCAN_LIBRARY") or LIB_PATH
        if p == LIB_PATH and not os.path.exists(p):
            from ._build import build
            build()
        if not os.path.exists(p):
            raise RuntimeError(f"libsscan.so not found at {p}; run __graft_entry__.build()")
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def lib():
    return _lib if _lib is not None else load_library()


def status_string(status: int) -> str:
    return lib().sscan_status_string(int(status)).decode()


def get_last_error() -> int:
    return int(lib().sscan_get_last_error())


def max_dstate() -> int:
    return int(lib().sscan_max_dstate())


def probe_ex2(blocks: int, iters: int, *, sink=None, stream=None) -> int:
    """Launch the exponent-unit throughput probe (see include/sscan.h) on the
    current device; returns the number of exponentials it computes.  Time it
    with CUDA events on ``stream``."""
    if sink is None:
        sink = torch.empty(blocks * 256, dtype=torch.float32, device="cuda")
    rc = lib().sscan_probe_ex2(_ptr(sink), int(blocks), int(iters), _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sscan_probe_ex2")
    return int(lib().sscan_probe_ex2_count(int(blocks), int(iters)))


def probe_element(blocks: int, iters: int, *, shared_rate: bool = False, sink=None, stream=None) -> int:
    """Launch the element-arithmetic throughput probe (see include/sscan.h) on
    the current device; returns the number of elements it computes.  Time it
    with CUDA events on ``stream``."""
    if sink is None:
        sink = torch.empty(blocks * 256, dtype=torch.float32, device="cuda")
    rc = lib().sscan_probe_element(_ptr(sink), int(blocks), int(iters), int(bool(shared_rate)),
                                   _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sscan_probe_element")
    return int(lib().sscan_probe_element_count(int(blocks), int(iters), int(bool(shared_rate))))


def debug_expire_next_wait(wait_limit_us: int) -> None:
    """Test aid: make the bounded waits of this thread's next forward call
    run out after ``wait_limit_us`` (see include/sscan.h)."""
    lib().sscan_debug_expire_next_wait(int(wait_limit_us))


def debug_expire_next_correction_wait(wait_limit_us: int) -> None:
    """Test aid: make the bounded waits of the carry correction of this
    thread's next forward call run out after ``wait_limit_us`` (see
    include/sscan.h)."""
    lib().sscan_debug_expire_next_correction_wait(int(wait_limit_us))


def last_launch_count() -> int:
    return int(lib().sscan_last_launch_count())


def last_plan() -> str:
    return lib().sscan_last_plan().decode()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(stream):
    if stream is None:  # the current stream of the current device, without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _check(t, name, shape, dtype, device):
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32


def _check_all(device, *tensors):
    """:func:`_check` of several (tensor, name, shape, dtype); None tensors pass."""
    for t, name, shape, dtype in tensors:
        if t is None or (t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous()):
            continue
        _check(t, name, shape, dtype, device)


def sscan_fwd(u, delta, A, B, C, D=None, h0=None, *, z=None, delta_bias=None,
              delta_softplus: bool = False, zoh: bool = False, out=None, final_state=None,
              return_final_state: bool = True, segments: int = 0, lanes: int = 0,
              stream=None):
    """Selective-scan forward on the GPU.  See the module docstring.

    Options (all inside the same kernels): ``delta_bias`` [dim] float32 is
    added to delta, ``delta_softplus`` then applies softplus to it, ``zoh``
    uses the zero-order-hold B-bar, and ``z`` [batch, dim, L] (I/O dtype)
    gates the output: out = (y + D*u) * silu(z).

    ``segments`` / ``lanes`` pin the launch plan (0 = automatic); the result is
    the same computation under any plan.  Returns ``(y, final_state)``
    (``final_state`` is None when ``return_final_state`` is False and none was
    passed).
    """
    if u.dim() != 3:
        raise ValueError("u must be [batch, dim, L]")
    batch, dim, L = u.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be [dim, N]")
    N = A.shape[1]
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan_fwd runs on CUDA tensors only")
    io = u.dtype
    if io not in (torch.float32, torch.bfloat16):
        raise ValueError("u must be float32 or bfloat16")
    _check(u, "u", (batch, dim, L), io, dev)
    _check(delta, "delta", (batch, dim, L), io, dev)
    _check(A, "A", (dim, N), torch.float32, dev)
    _check(B, "B", (batch, N, L), io, dev)
    _check(C, "C", (batch, N, L), io, dev)
    if D is not None:
        _check(D, "D", (dim,), torch.float32, dev)
    if h0 is not None:
        _check(h0, "h0", (batch, dim, N), torch.float32, dev)
    if z is not None:
        _check(z, "z", (batch, dim, L), io, dev)
    if delta_bias is not None:
        _check(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    if out is None:
        out = torch.empty((batch, dim, L), dtype=io, device=dev)
    else:
        _check(out, "out", (batch, dim, L), io, dev)
    if final_state is None and return_final_state:
        final_state = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    elif final_state is not None:
        _check(final_state, "final_state", (batch, dim, N), torch.float32, dev)
    dtype = SSCAN_F32 if io == torch.float32 else SSCAN_BF16
    flags = (SSCAN_DELTA_SOFTPLUS if delta_softplus else 0) | (SSCAN_ZOH if zoh else 0)
    if z is None and delta_bias is None and flags == 0:
        rc = lib().sscan_fwd_ex(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                _ptr(h0), _ptr(out), _ptr(final_state), batch, dim, L, N,
                                dtype, int(segments), int(lanes), _stream_handle(stream))
    else:
        rc = lib().sscan_fwd_fused(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                   _ptr(z), _ptr(delta_bias), _ptr(h0), _ptr(out),
                                   _ptr(final_state), batch, dim, L, N, dtype, flags,
                                   int(segments), int(lanes), _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sscan_fwd")
    return out, final_state


def sscan_bwd(u, delta, A, B, C, D, h0, dy, dfinal_state=None, *, stream=None):
    """Gradients of :func:`sscan_fwd` (no options) for upstream gradients ``dy``
    [batch, dim, L] (I/O dtype) and ``dfinal_state`` [batch, dim, N] float32
    (None = 0).  Returns a dict with du, ddelta (I/O dtype), dA, dB, dC, dD (None
    when D is None) and dh0 (float32)."""
    if u.dim() != 3:
        raise ValueError("u must be [batch, dim, L]")
    batch, dim, L = u.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be [dim, N]")
    N = A.shape[1]
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan_bwd runs on CUDA tensors only")
    io = u.dtype
    if io not in (torch.float32, torch.bfloat16):
        raise ValueError("u must be float32 or bfloat16")
    for t, name, shape, dt in ((u, "u", (batch, dim, L), io), (delta, "delta", (batch, dim, L), io),
                               (A, "A", (dim, N), torch.float32), (B, "B", (batch, N, L), io),
                               (C, "C", (batch, N, L), io), (dy, "dy", (batch, dim, L), io)):
        _check(t, name, shape, dt, dev)
    if D is not None:
        _check(D, "D", (dim,), torch.float32, dev)
    if h0 is not None:
        _check(h0, "h0", (batch, dim, N), torch.float32, dev)
    if dfinal_state is not None:
        _check(dfinal_state, "dfinal_state", (batch, dim, N), torch.float32, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"du": torch.empty((batch, dim, L), dtype=io, device=dev),
         "ddelta": torch.empty((batch, dim, L), dtype=io, device=dev),
         "dA": torch.empty((dim, N), **f32), "dB": torch.empty((batch, N, L), **f32),
         "dC": torch.empty((batch, N, L), **f32),
         "dD": None if D is None else torch.empty((dim,), **f32),
         "dh0": torch.empty((batch, dim, N), **f32)}
    dtype = SSCAN_F32 if io == torch.float32 else SSCAN_BF16
    rc = lib().sscan_bwd(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(h0), _ptr(dy),
                         _ptr(dfinal_state), _ptr(g["du"]), _ptr(g["ddelta"]), _ptr(g["dA"]),
                         _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["dh0"]),
                         batch, dim, L, N, dtype, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sscan_bwd")
    return g


def sscan_step(u, delta, A, B, C, D=None, *, state, slots=None, z=None, delta_bias=None,
               delta_softplus: bool = False, out=None, stream=None):
    """One decode step: advances ``state`` [batch, dim, N] (float32, in place)
    by one token and returns y [batch, dim].  u, delta: [batch, dim]; B, C:
    [batch, N] (float32 or bfloat16, like u); A [dim, N] and D [dim] float32.

    ``slots`` [batch] int32 makes ``state`` a cache [rows, dim, N] of which
    request b uses row ``slots[b]`` (distinct rows; negative: padding that
    starts from zeros and keeps no state).  ``delta_bias`` [dim] float32,
    ``delta_softplus`` and the gate ``z`` [batch, dim] (unit channel stride) act as in
    :func:`sscan_fwd`."""
    if u.dim() != 2:
        raise ValueError("u must be [batch, dim]")
    batch, dim = u.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be [dim, N]")
    N = A.shape[1]
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan_step runs on CUDA tensors only")
    io = u.dtype
    if io not in (torch.float32, torch.bfloat16):
        raise ValueError("u must be float32 or bfloat16")
    rows = state.shape[0] if slots is not None and state.dim() == 3 else batch
    each, few = (batch, dim), (batch, N)
    _check_all(dev, (u, "u", each, io), (delta, "delta", each, io), (A, "A", (dim, N), _F32), (B, "B", few, io),
               (C, "C", few, io), (D, "D", (dim,), _F32), (state, "state", (rows, dim, N), _F32),
               (slots, "slots", (batch,), _I32), (delta_bias, "delta_bias", (dim,), _F32))
    if z is not None:
        _check_rows(z, "z", each, io, dev)
    if out is None:
        out = torch.empty_like(u)
    else:
        _check(out, "out", (batch, dim), io, dev)
    dtype = SSCAN_F32 if io == torch.float32 else SSCAN_BF16
    if slots is None and z is None and delta_bias is None and not delta_softplus:  # as before the options: the same bits
        rc = lib().sscan_step(u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), state.data_ptr(),
                              out.data_ptr(), batch, dim, N, dtype, _stream_handle(stream))
    else:
        rc = lib().sscan_step_slots(u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z),
                                    _ptr(delta_bias), _ptr(slots), state.data_ptr(), out.data_ptr(), batch, rows, dim, N,
                                    0 if z is None else z.stride(0), dtype,
                                    SSCAN_DELTA_SOFTPLUS if delta_softplus else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sscan_step")
    return out


def _check_rows(t, name, shape, dtype, device):
    """As :func:`_check`, but only the last dimension has to be contiguous (the
    tensor may be a view, such as one half of a joint projection)."""
    if t.shape == shape and t.dtype is dtype and t.device == device and (t.stride(-1) == 1 or shape[-1] <= 1):
        return
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _io(t, name, dims, where):
    """The dtype code of an I/O tensor with ``dims`` dimensions on the GPU."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{where} runs on CUDA tensors only")
    if t.dtype is _F32:
        return SSCAN_F32
    if t.dtype is _BF16:
        return SSCAN_BF16
    raise ValueError(f"{name} must be float32 or bfloat16")


def _check_tables(cu_seqlens, slots, has_state, state, rest, dtype, dev):
    """Check a packed call's request tables and cache; returns the number of requests."""
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [requests + 1]")
    n = cu_seqlens.shape[0] - 1
    if state.dim() != 3:
        raise ValueError("state must have 3 dimensions")
    rows = state.shape[0]
    _check_all(dev, (cu_seqlens, "cu_seqlens", (n + 1,), _I32), (slots, "slots", (n,), _I32),
               (has_state, "has_state", (n,), torch.bool), (state, "state", (rows, *rest), dtype))
    if slots is None and n > rows:
        raise ValueError(f"state has {rows} rows for {n} requests")
    return n


def _sconv_weight(weight, bias, dim, dev):
    if weight.dim() != 2 or weight.shape[0] != dim:
        raise ValueError("weight must be [dim, width]")
    width = weight.shape[1]
    if not 2 <= width <= SCONV_MAX_WIDTH:
        raise ValueError(f"weight must have 2 to {SCONV_MAX_WIDTH} taps, got {width}")
    _check_all(dev, (weight, "weight", (dim, width), _F32), (bias, "bias", (dim,), _F32))
    return width


def sconv_fwd(x, weight, bias=None, x0=None, *, silu: bool = True, out=None, final_state=None,
              return_final_state: bool = True, stream=None):
    """Short causal depthwise convolution before the scan, with SiLU (see
    include/sscan.h): x [batch, dim, L] (float32 or bfloat16; a view with unit
    time stride will do), weight [dim, W] and bias [dim] float32 with W = 2 to
    4, x0 [batch, dim, W-1] the inputs before the first (None = zeros).
    Returns ``(y, final_state)``; final_state [batch, dim, W-1], the last W-1
    inputs, is None when ``return_final_state`` is False and none was passed."""
    dtype = _io(x, "x", 3, "sconv_fwd")
    batch, dim, L = x.shape
    dev, io = x.device, x.dtype
    _check_rows(x, "x", (batch, dim, L), io, dev)
    width = _sconv_weight(weight, bias, dim, dev)
    tail = (batch, dim, width - 1)
    if x0 is not None:
        _check(x0, "x0", tail, io, dev)
    if out is None:
        out = torch.empty((batch, dim, L), dtype=io, device=dev)
    else:
        _check(out, "out", (batch, dim, L), io, dev)
    if final_state is not None:
        _check(final_state, "final_state", tail, io, dev)
    elif return_final_state:
        final_state = torch.empty(tail, dtype=io, device=dev)
    rc = lib().sconv_fwd(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(x0), out.data_ptr(), _ptr(final_state), batch, dim, L,
                         width, x.stride(0), x.stride(1), dtype, SCONV_SILU if silu else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sconv_fwd")
    return out, final_state


def sconv_bwd(x, weight, bias, x0, dy, dfinal_state=None, *, silu: bool = True, stream=None):
    """Gradients of :func:`sconv_fwd` for upstream gradients ``dy`` [batch, dim, L]
    and ``dfinal_state`` [batch, dim, W-1] (I/O dtype; None = 0).  Returns a dict
    with dx, dx0 (I/O dtype; dx0 None when x0 is), dweight and dbias (float32;
    dbias None when bias is)."""
    dtype = _io(x, "x", 3, "sconv_bwd")
    batch, dim, L = x.shape
    dev, io = x.device, x.dtype
    _check_rows(x, "x", (batch, dim, L), io, dev)
    width = _sconv_weight(weight, bias, dim, dev)
    tail = (batch, dim, width - 1)
    _check(dy, "dy", (batch, dim, L), io, dev)
    if x0 is not None:
        _check(x0, "x0", tail, io, dev)
    if dfinal_state is not None:
        _check(dfinal_state, "dfinal_state", tail, io, dev)
    g = {"dx": torch.empty((batch, dim, L), dtype=io, device=dev),
         "dweight": torch.empty((dim, width), dtype=torch.float32, device=dev),
         "dbias": None if bias is None else torch.empty((dim,), dtype=torch.float32, device=dev),
         "dx0": None if x0 is None else torch.empty(tail, dtype=io, device=dev)}
    rc = lib().sconv_bwd(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(x0), dy.data_ptr(), _ptr(dfinal_state), g["dx"].data_ptr(),
                         g["dweight"].data_ptr(), _ptr(g["dbias"]), _ptr(g["dx0"]), batch, dim, L, width, x.stride(0),
                         x.stride(1), dtype, SCONV_SILU if silu else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sconv_bwd")
    return g


def sconv_prompt(x, weight, bias=None, *, cu_seqlens, state, slots=None, has_state=None, silu: bool = True,
                 out=None, stream=None):
    """:func:`sconv_fwd` on packed prompts over a cache: x [dim, tokens] (unit
    time stride), request s owning tokens ``cu_seqlens[s]`` to ``cu_seqlens[s+1]``
    (int32) and row ``slots[s]`` (int32; None: row s; negative: keeps no state)
    of ``state`` [rows, dim, W-1] (I/O dtype), which is updated in place.
    ``has_state`` [requests] bool: continue from the row, or from zeros (None:
    all continue).  Returns y [dim, tokens]."""
    dtype = _io(x, "x", 2, "sconv_prompt")
    dim, tokens = x.shape
    dev, io = x.device, x.dtype
    _check_rows(x, "x", (dim, tokens), io, dev)
    width = _sconv_weight(weight, bias, dim, dev)
    n = _check_tables(cu_seqlens, slots, has_state, state, (dim, width - 1), io, dev)
    if out is None:
        out = torch.empty((dim, tokens), dtype=io, device=dev)
    else:
        _check(out, "out", (dim, tokens), io, dev)
    rc = lib().sconv_prompt(x.data_ptr(), weight.data_ptr(), _ptr(bias), cu_seqlens.data_ptr(), _ptr(slots), _ptr(has_state),
                            state.data_ptr(), out.data_ptr(), n, state.shape[0], dim, tokens, width, x.stride(0), dtype,
                            SCONV_SILU if silu else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sconv_prompt")
    return out


def sconv_step(x, weight, bias=None, *, state, slots=None, silu: bool = True, out=None, stream=None):
    """One token of every request: x [batch, dim] (unit channel stride), ``state``
    [rows, dim, W-1] (I/O dtype) updated in place, ``slots`` as in
    :func:`sconv_prompt`.  Returns y [batch, dim]."""
    dtype = _io(x, "x", 2, "sconv_step")
    batch, dim = x.shape
    dev, io = x.device, x.dtype
    _check_rows(x, "x", (batch, dim), io, dev)
    width = _sconv_weight(weight, bias, dim, dev)
    if state.dim() != 3:
        raise ValueError("state must have 3 dimensions")
    rows = state.shape[0] if slots is not None else batch
    _check_all(dev, (state, "state", (rows, dim, width - 1), io), (slots, "slots", (batch,), _I32))
    if out is None:
        out = torch.empty((batch, dim), dtype=io, device=dev)
    else:
        _check(out, "out", (batch, dim), io, dev)
    rc = lib().sconv_step(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(slots), state.data_ptr(), out.data_ptr(), batch, rows, dim,
                          width, x.stride(0), dtype, SCONV_SILU if silu else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sconv_step")
    return out


def sscan_prompt(u, delta, A, B, C, D=None, *, cu_seqlens, state, slots=None, has_state=None, z=None,
                 delta_bias=None, delta_softplus: bool = False, out=None, segments: int = 0, stream=None):
    """Selective scan of packed prompts over a state cache: u, delta (and the
    gate z) [dim, tokens], B, C [N, tokens], ``state`` [rows, dim, N] float32
    updated in place; the request tables are those of :func:`sconv_prompt`, the
    options those of :func:`sscan_fwd`.  ``segments`` pins the number of pieces
    that the packed axis is cut into (0 = automatic); the result is the same
    computation under any, but for what has decayed below 2^-26 of its size
    when it entered before a piece's border, which is left out there.  Step
    sizes must not be negative.  Returns y [dim, tokens]."""
    dtype = _io(u, "u", 2, "sscan_prompt")
    dim, tokens = u.shape
    dev, io = u.device, u.dtype
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be [dim, N]")
    N = A.shape[1]
    each, few = (dim, tokens), (N, tokens)
    _check_all(dev, (u, "u", each, io), (delta, "delta", each, io), (A, "A", (dim, N), _F32), (B, "B", few, io),
               (C, "C", few, io), (D, "D", (dim,), _F32), (z, "z", each, io), (delta_bias, "delta_bias", (dim,), _F32))
    n = _check_tables(cu_seqlens, slots, has_state, state, (dim, N), _F32, dev)
    if out is None:
        out = torch.empty_like(u)
    else:
        _check(out, "out", (dim, tokens), io, dev)
    rc = lib().sscan_prompt(u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z), _ptr(delta_bias),
                            cu_seqlens.data_ptr(), _ptr(slots), _ptr(has_state), state.data_ptr(), out.data_ptr(), n,
                            state.shape[0], dim, tokens, N, dtype, SSCAN_DELTA_SOFTPLUS if delta_softplus else 0,
                            int(segments), _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "sscan_prompt")
    return out


def addnorm_fwd(x, residual, weight, *, scale: float = 1.0, eps: float = 1e-5, out=None, residual_out=None,
                stream=None):
    """RMS norm before a layer, fused with the residual addition: r = residual +
    scale*x, y = r / sqrt(mean(r^2) + eps) * weight.  x [rows, width] (float32
    or bfloat16), residual [rows, width] float32 (None = 0), weight [width]
    float32.  Returns ``(y, r)``; r is float32 and may be written over
    ``residual`` (``residual_out=residual``)."""
    dtype = _io(x, "x", 2, "addnorm_fwd")
    rows, width = x.shape
    dev, io = x.device, x.dtype
    each = (rows, width)
    _check_all(dev, (x, "x", each, io), (weight, "weight", (width,), _F32), (residual, "residual", each, _F32))
    if out is None:
        out = torch.empty_like(x)
    else:
        _check(out, "out", (rows, width), io, dev)
    if residual_out is None:
        residual_out = torch.empty(each, dtype=_F32, device=dev)
    else:
        _check(residual_out, "residual_out", (rows, width), torch.float32, dev)
    rc = lib().addnorm_fwd(x.data_ptr(), _ptr(residual), weight.data_ptr(), out.data_ptr(), residual_out.data_ptr(), rows, width,
                           scale, eps, dtype, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "addnorm_fwd")
    return out, residual_out


def addnorm_bwd(residual_out, weight, dy, dresidual_out=None, *, scale: float = 1.0, eps: float = 1e-5, stream=None):
    """Gradients of :func:`addnorm_fwd` from its ``residual_out``, for upstream
    gradients ``dy`` [rows, width] (I/O dtype) and ``dresidual_out`` [rows, width]
    float32 (None = 0).  Returns a dict with dx (I/O dtype), dresidual and
    dweight (float32)."""
    dtype = _io(dy, "dy", 2, "addnorm_bwd")
    rows, width = dy.shape
    dev, io = dy.device, dy.dtype
    _check(dy, "dy", (rows, width), io, dev)
    _check(residual_out, "residual_out", (rows, width), torch.float32, dev)
    _check(weight, "weight", (width,), torch.float32, dev)
    if dresidual_out is not None:
        _check(dresidual_out, "dresidual_out", (rows, width), torch.float32, dev)
    g = {"dx": torch.empty((rows, width), dtype=io, device=dev),
         "dresidual": torch.empty((rows, width), dtype=torch.float32, device=dev),
         "dweight": torch.empty((width,), dtype=torch.float32, device=dev)}
    rc = lib().addnorm_bwd(residual_out.data_ptr(), weight.data_ptr(), dy.data_ptr(), _ptr(dresidual_out), g["dx"].data_ptr(),
                           g["dresidual"].data_ptr(), g["dweight"].data_ptr(), rows, width, scale, eps, dtype,
                           _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "addnorm_bwd")
    return g


def _gatenorm_args(y, z, weight, groups, dims, where):
    dtype = _io(y, "y", dims, where)
    dev, io, shape = y.device, y.dtype, y.shape
    dim = shape[1]
    _check_all(dev, (y, "y", shape, io), (weight, "weight", (dim,), _F32))
    _check_rows(z, "z", shape, io, dev)
    if groups < 1 or dim % groups != 0:
        raise ValueError(f"groups must divide the {dim} channels, got {groups}")
    return dtype


def gatenorm_fwd(y, z, weight, *, groups: int = 1, norm_first: bool = False, eps: float = 1e-5, out=None,
                 stream=None):
    """Gated RMS norm after the scan, over the channels of y [batch, dim, L] in
    ``groups`` equal parts: with v = y * silu(z), v / sqrt(mean(v^2) + eps) *
    weight; with ``norm_first`` the norm of y times weight and silu(z).  z may be
    a view with unit time stride; weight [dim] float32.  Returns out [batch, dim, L]."""
    dtype = _gatenorm_args(y, z, weight, groups, 3, "gatenorm_fwd")
    if out is None:
        out = torch.empty_like(y)
    else:
        _check(out, "out", y.shape, y.dtype, y.device)
    batch, dim, L = y.shape
    rc = lib().gatenorm_fwd(y.data_ptr(), _ptr(z), weight.data_ptr(), out.data_ptr(), batch, dim, L, groups, z.stride(0), z.stride(1),
                            eps, dtype, GATENORM_NORM_FIRST if norm_first else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "gatenorm_fwd")
    return out


def gatenorm_bwd(y, z, weight, dout, *, groups: int = 1, norm_first: bool = False, eps: float = 1e-5, stream=None):
    """Gradients of :func:`gatenorm_fwd` for the upstream gradient ``dout``
    [batch, dim, L].  Returns a dict with dy, dz (I/O dtype) and dweight (float32)."""
    dtype = _gatenorm_args(y, z, weight, groups, 3, "gatenorm_bwd")
    _check(dout, "dout", y.shape, y.dtype, y.device)
    batch, dim, L = y.shape
    g = {"dy": torch.empty_like(y), "dz": torch.empty_like(y),
         "dweight": torch.empty((dim,), dtype=torch.float32, device=y.device)}
    rc = lib().gatenorm_bwd(y.data_ptr(), _ptr(z), weight.data_ptr(), dout.data_ptr(), g["dy"].data_ptr(), g["dz"].data_ptr(),
                            g["dweight"].data_ptr(), batch, dim, L, groups, z.stride(0), z.stride(1), eps, dtype,
                            GATENORM_NORM_FIRST if norm_first else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "gatenorm_bwd")
    return g


def gatenorm_step(y, z, weight, *, groups: int = 1, norm_first: bool = False, eps: float = 1e-5, out=None,
                  stream=None):
    """:func:`gatenorm_fwd` of single tokens: y, z [rows, dim] (z with unit channel
    stride).  Returns out [rows, dim]."""
    dtype = _gatenorm_args(y, z, weight, groups, 2, "gatenorm_step")
    if out is None:
        out = torch.empty_like(y)
    else:
        _check(out, "out", y.shape, y.dtype, y.device)
    rows, dim = y.shape
    rc = lib().gatenorm_step(y.data_ptr(), _ptr(z), weight.data_ptr(), out.data_ptr(), rows, dim, groups, z.stride(0), eps, dtype,
                             GATENORM_NORM_FIRST if norm_first else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "gatenorm_step")
    return out


def pscan(a, b, h0=None, *, out=None, stream=None):
    """h[r,t] = a[r,t]*h[r,t-1] + b[r,t] with h[r,-1] = h0[r] (0 if None), on
    float32 CUDA tensors a, b [rows, len].  Returns h [rows, len]."""
    if a.dim() != 2:
        raise ValueError("a must be [rows, len]")
    rows, n = a.shape
    dev = a.device
    if dev.type != "cuda":
        raise ValueError("pscan runs on CUDA tensors only")
    _check(a, "a", (rows, n), torch.float32, dev)
    _check(b, "b", (rows, n), torch.float32, dev)
    if h0 is not None:
        _check(h0, "h0", (rows,), torch.float32, dev)
    if out is None:
        out = torch.empty((rows, n), dtype=torch.float32, device=dev)
    else:
        _check(out, "out", (rows, n), torch.float32, dev)
    rc = lib().pscan(_ptr(a), _ptr(b), _ptr(out), _ptr(h0), rows, n, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "pscan")
    return out


_I64x4, _I64x8 = ctypes.c_int64 * 4, ctypes.c_int64 * 8


def _on_current(dev, where):
    """The launch goes to the current device's stream: its tensors have to lie there."""
    if dev.index != torch._C._cuda_getDevice():
        raise ValueError(f"{where}: tensors are on {dev}, the current device is cuda:{torch._C._cuda_getDevice()}")


def _lattn_shapes(q, k, v, A, delta, D, delta_bias, groups, dims, where):
    """Check the inputs that the lattn calls share; ``dims`` is 3 ([batch, channels,
    L]) or 2 (packed [channels, tokens], or single tokens [batch, channels] when
    ``where`` is lattn_step).  Returns (dtype, heads, key, value channels)."""
    dtype = _io(v, "v", dims, where)
    dev, io = v.device, v.dtype
    at = 0 if where == "lattn_prompt" else 1  # the channels' dimension
    if A.dim() != 1:
        raise ValueError("A must be [heads]")
    heads, dim = A.shape[0], v.shape[at]
    if heads < 1 or dim % heads or not 1 <= dim // heads <= LATTN_MAX_VALUE:
        raise ValueError(f"v must have heads * (1 to {LATTN_MAX_VALUE}) channels, got {dim} for {heads} heads")
    if q.dim() != dims:
        raise ValueError(f"q must have {dims} dimensions, got {q.dim()}")
    groups = int(groups)
    if groups < 1 or heads % groups or q.shape[at] % groups or not 1 <= q.shape[at] // groups <= LATTN_MAX_KEY:
        raise ValueError(f"q must have groups * (1 to {LATTN_MAX_KEY}) channels and groups must divide the {heads} heads, "
                         f"got {q.shape[at]} channels and {groups} groups")
    lead, tail = tuple(v.shape[:at]), tuple(v.shape[at + 1:])
    few, rows = lead + (q.shape[at],) + tail, lead + (heads,) + tail
    _check_rows(v, "v", tuple(v.shape), io, dev)
    _check_rows(q, "q", few, io, dev)
    _check_rows(k, "k", few, io, dev)
    if delta is not None:
        _check_rows(delta, "delta", rows, io, dev)
    elif delta_bias is not None:
        raise ValueError("delta_bias needs delta")
    _check_all(dev, (A, "A", (heads,), _F32), (D, "D", (heads,), _F32), (delta_bias, "delta_bias", (heads,), _F32))
    _on_current(dev, where)
    return dtype, heads, q.shape[at] // groups, dim // heads


def _batch_strides(q, k, v, delta):
    return _I64x8(q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                  *((0, 0) if delta is None else (delta.stride(0), delta.stride(1))))


def lattn_fwd(q, k, v, A, delta=None, D=None, s0=None, *, groups: int = 1, scale: float = 1.0, delta_bias=None,
              delta_softplus: bool = False, out=None, final_state=None, return_final_state: bool = True, pieces: int = 0,
              stream=None):
    """Linear attention with a decay for each head (see include/sscan.h):
    S_t = exp(A dt_t) S_{t-1} + dt_t v_t k_t^T, o_t = scale * S_t q_t + D v_t.

    v [batch, heads*P, L], q and k [batch, groups*N, L] (float32 or bfloat16;
    views with unit time stride will do), A and D [heads] float32, ``delta``
    [batch, heads, L] the steps dt (like v; None: steps of one), after
    ``delta_bias`` [heads] float32 and softplus where asked for; s0 [batch, heads*P, N]
    float32 (None = zeros).  ``groups`` sets of queries and keys are shared by equal
    numbers of consecutive heads.  ``pieces`` pins the number of parts of time that
    run side by side (0 = automatic).  Returns ``(o, final_state)``; final_state
    is None when ``return_final_state`` is False and none was passed."""
    dtype, heads, key, value = _lattn_shapes(q, k, v, A, delta, D, delta_bias, groups, 3, "lattn_fwd")
    batch, dim, L = v.shape
    dev, io = v.device, v.dtype
    states = (batch, dim, key)
    _check_all(dev, (s0, "s0", states, _F32), (out, "out", (batch, dim, L), io), (final_state, "final_state", states, _F32))
    if out is None:
        out = torch.empty((batch, dim, L), dtype=io, device=dev)
    if final_state is None and return_final_state:
        final_state = torch.empty(states, dtype=_F32, device=dev)
    rc = lib().lattn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), A.data_ptr(), _ptr(delta), _ptr(D), _ptr(delta_bias), _ptr(s0),
                         out.data_ptr(), _ptr(final_state), batch, heads, int(groups), key, value, L, _batch_strides(q, k, v, delta),
                         scale, dtype, SSCAN_DELTA_SOFTPLUS if delta_softplus else 0, int(pieces), _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "lattn_fwd")
    return out, final_state


def lattn_bwd(q, k, v, A, delta, D, s0, do, dfinal_state=None, *, groups: int = 1, scale: float = 1.0, delta_bias=None,
              delta_softplus: bool = False, stream=None):
    """Gradients of :func:`lattn_fwd` for upstream gradients ``do`` [batch, heads*P, L]
    (I/O dtype) and ``dfinal_state`` [batch, heads*P, N] float32 (None = 0).
    Returns a dict with dq, dk, dv and ddelta (I/O dtype; dq and dk summed over the heads
    that share them), dA, dD, ddelta_bias and ds0 (float32); ddelta, dD, ddelta_bias
    and ds0 are None when their input is."""
    dtype, heads, key, value = _lattn_shapes(q, k, v, A, delta, D, delta_bias, groups, 3, "lattn_bwd")
    batch, dim, L = v.shape
    dev, io = v.device, v.dtype
    states = (batch, dim, key)
    _check_all(dev, (s0, "s0", states, _F32), (do, "do", (batch, dim, L), io), (dfinal_state, "dfinal_state", states, _F32))
    f32 = dict(dtype=_F32, device=dev)
    like = dict(dtype=io, device=dev)
    g = {"dq": torch.empty(q.shape, **like), "dk": torch.empty(k.shape, **like), "dv": torch.empty(v.shape, **like),
         "ddelta": None if delta is None else torch.empty((batch, heads, L), **like), "dA": torch.empty((heads,), **f32),
         "dD": None if D is None else torch.empty((heads,), **f32),
         "ddelta_bias": None if delta_bias is None else torch.empty((heads,), **f32),
         "ds0": None if s0 is None else torch.empty(states, **f32)}
    rc = lib().lattn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), A.data_ptr(), _ptr(delta), _ptr(D), _ptr(delta_bias), _ptr(s0),
                         do.data_ptr(), _ptr(dfinal_state), g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(),
                         _ptr(g["ddelta"]), g["dA"].data_ptr(), _ptr(g["dD"]), _ptr(g["ddelta_bias"]), _ptr(g["ds0"]), batch, heads,
                         int(groups), key, value, L, _batch_strides(q, k, v, delta), scale, dtype,
                         SSCAN_DELTA_SOFTPLUS if delta_softplus else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "lattn_bwd")
    return g


def lattn_prompt(q, k, v, A, delta=None, D=None, *, cu_seqlens, state, slots=None, has_state=None, groups: int = 1,
                 scale: float = 1.0, delta_bias=None, delta_softplus: bool = False, out=None, pieces: int = 0, stream=None):
    """:func:`lattn_fwd` on packed prompts over a state cache: q, k [groups*N,
    tokens], v [heads*P, tokens], delta [heads, tokens] (unit time stride),
    ``state`` [rows, heads*P, N] float32 updated in place; the request tables are
    those of :func:`sconv_prompt`.  Returns o [heads*P, tokens]."""
    dtype, heads, key, value = _lattn_shapes(q, k, v, A, delta, D, delta_bias, groups, 2, "lattn_prompt")
    dim, tokens = v.shape
    dev, io = v.device, v.dtype
    n = _check_tables(cu_seqlens, slots, has_state, state, (dim, key), _F32, dev)
    if out is None:
        out = torch.empty((dim, tokens), dtype=io, device=dev)
    else:
        _check(out, "out", (dim, tokens), io, dev)
    strides = _I64x8(0, q.stride(0), 0, k.stride(0), 0, v.stride(0), 0, 0 if delta is None else delta.stride(0))
    rc = lib().lattn_prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), A.data_ptr(), _ptr(delta), _ptr(D), _ptr(delta_bias),
                            cu_seqlens.data_ptr(), _ptr(slots), _ptr(has_state), state.data_ptr(), out.data_ptr(), n, state.shape[0],
                            heads, int(groups), key, value, tokens, strides, scale, dtype,
                            SSCAN_DELTA_SOFTPLUS if delta_softplus else 0, int(pieces), _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "lattn_prompt")
    return out


def lattn_step(q, k, v, A, delta=None, D=None, *, state, slots=None, groups: int = 1, scale: float = 1.0, delta_bias=None,
               delta_softplus: bool = False, out=None, stream=None):
    """One token of every request through :func:`lattn_fwd`: q, k [batch,
    groups*N], v [batch, heads*P], delta [batch, heads] (unit channel stride), ``state``
    [rows, heads*P, N] float32 updated in place, ``slots`` as in
    :func:`sconv_prompt`.  Returns o [batch, heads*P]."""
    dtype, heads, key, value = _lattn_shapes(q, k, v, A, delta, D, delta_bias, groups, 2, "lattn_step")
    batch, dim = v.shape
    dev, io = v.device, v.dtype
    if state.dim() != 3:
        raise ValueError("state must have 3 dimensions")
    rows = state.shape[0] if slots is not None else batch
    _check_all(dev, (state, "state", (rows, dim, key), _F32), (slots, "slots", (batch,), _I32), (out, "out", (batch, dim), io))
    if out is None:
        out = torch.empty((batch, dim), dtype=io, device=dev)
    rc = lib().lattn_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), A.data_ptr(), _ptr(delta), _ptr(D), _ptr(delta_bias), _ptr(slots),
                          state.data_ptr(), out.data_ptr(), batch, rows, heads, int(groups), key, value, q.stride(0), k.stride(0),
                          v.stride(0), 0 if delta is None else delta.stride(0), scale, dtype,
                          SSCAN_DELTA_SOFTPLUS if delta_softplus else 0, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "lattn_step")
    return out


def _qk_shapes(q, k, q_weight, k_weight, positions, inv_freq, dims, where):
    """Check the inputs that the qknorm calls share.  Returns (dtype, head width, query
    heads, key heads, frequencies)."""
    dtype = _io(q, "q", dims, where)
    dev, io = q.device, q.dtype
    if q_weight.dim() != 1 or not 1 <= q_weight.shape[0] <= QKNORM_MAX_DIM:
        raise ValueError(f"q_weight must be [1 to {QKNORM_MAX_DIM}]")
    width = q_weight.shape[0]
    _check_all(dev, (q_weight, "q_weight", (width,), _F32), (k_weight, "k_weight", (width,), _F32))
    if (k is None) != (k_weight is None):
        raise ValueError("k and k_weight go together")
    lead, tail = tuple(q.shape[:1]), tuple(q.shape[2:])
    for t, name in ((q, "q"), (k, "k")):
        if t is None:
            continue
        if t.dim() != dims or t.shape[1] % width:
            raise ValueError(f"{name} must have {dims} dimensions and heads * {width} channels, got {tuple(t.shape)}")
        _check_rows(t, name, lead + (t.shape[1],) + tail, io, dev)
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    rotated = 0
    if inv_freq is not None:
        rotated = inv_freq.shape[0] if inv_freq.dim() == 1 else -1
        if not 1 <= rotated <= width // 2:
            raise ValueError(f"inv_freq must be [1 to {width // 2}], got {tuple(inv_freq.shape)}")
        _check_all(dev, (positions, "positions", lead + tail, _I32), (inv_freq, "inv_freq", (rotated,), _F32))
    _on_current(dev, where)
    return dtype, width, q.shape[1] // width, 0 if k is None else k.shape[1] // width, rotated


def qknorm_fwd(q, k, q_weight, k_weight, positions=None, inv_freq=None, *, eps: float = 1e-5, out=None, stream=None):
    """RMS norms of queries and keys for each head and their rotation by position,
    in one pass (see include/sscan.h): q [batch, q_heads*D, L], k [batch, k_heads*D,
    L] (float32 or bfloat16; views with unit time stride will do), weights [D] float32,
    ``positions`` [batch, L] int32 and ``inv_freq`` [r] float32: channels i and i + r
    of a head turn by positions * inv_freq[i] (None: no rotation).  k and k_weight may be
    None.  ``out``: a pair of tensors to write.  Returns ``(q_out, k_out)``."""
    dtype, width, qh, kh, rotated = _qk_shapes(q, k, q_weight, k_weight, positions, inv_freq, 3, "qknorm_fwd")
    batch, _, L = q.shape
    dev, io = q.device, q.dtype
    if out is None:
        qo = torch.empty(q.shape, dtype=io, device=dev)
        ko = None if k is None else torch.empty(k.shape, dtype=io, device=dev)
    else:
        qo, ko = out
        _check_all(dev, (qo, "out[0]", q.shape, io), (ko, "out[1]", q.shape if k is None else k.shape, io))
        if qo is None or (ko is None) != (k is None):
            raise ValueError("out must hold a tensor for q, and one for k where k is given")
    strides = _I64x4(q.stride(0), q.stride(1), *((0, 0) if k is None else (k.stride(0), k.stride(1))))
    rc = lib().qknorm_fwd(q.data_ptr(), _ptr(k), q_weight.data_ptr(), _ptr(k_weight), _ptr(positions), _ptr(inv_freq), qo.data_ptr(),
                          _ptr(ko), batch, qh, kh, width, L, rotated, strides, eps, dtype, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "qknorm_fwd")
    return qo, ko


def qknorm_bwd(q, k, q_weight, k_weight, dq_out, dk_out, positions=None, inv_freq=None, *, eps: float = 1e-5, stream=None):
    """Gradients of :func:`qknorm_fwd` for upstream gradients ``dq_out`` and
    ``dk_out`` (like q and k, contiguous).  Returns a dict with dq, dk (I/O dtype),
    dq_weight and dk_weight (float32); dk and dk_weight are None when k is."""
    dtype, width, qh, kh, rotated = _qk_shapes(q, k, q_weight, k_weight, positions, inv_freq, 3, "qknorm_bwd")
    batch, _, L = q.shape
    dev, io = q.device, q.dtype
    _check(dq_out, "dq_out", tuple(q.shape), io, dev)
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    if k is not None:
        _check(dk_out, "dk_out", tuple(k.shape), io, dev)
    g = {"dq": torch.empty(q.shape, dtype=io, device=dev), "dk": None if k is None else torch.empty(k.shape, dtype=io, device=dev),
         "dq_weight": torch.empty((width,), dtype=_F32, device=dev),
         "dk_weight": None if k is None else torch.empty((width,), dtype=_F32, device=dev)}
    strides = _I64x4(q.stride(0), q.stride(1), *((0, 0) if k is None else (k.stride(0), k.stride(1))))
    rc = lib().qknorm_bwd(q.data_ptr(), _ptr(k), q_weight.data_ptr(), _ptr(k_weight), _ptr(positions), _ptr(inv_freq), dq_out.data_ptr(),
                          _ptr(dk_out), g["dq"].data_ptr(), _ptr(g["dk"]), g["dq_weight"].data_ptr(), _ptr(g["dk_weight"]), batch, qh, kh,
                          width, L, rotated, strides, eps, dtype, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "qknorm_bwd")
    return g


def qknorm_step(q, k, q_weight, k_weight, positions=None, inv_freq=None, *, eps: float = 1e-5, out=None, stream=None):
    """:func:`qknorm_fwd` of single tokens: q [batch, q_heads*D], k [batch,
    k_heads*D] (unit channel stride), ``positions`` [batch]."""
    dtype, width, qh, kh, rotated = _qk_shapes(q, k, q_weight, k_weight, positions, inv_freq, 2, "qknorm_step")
    batch, dev, io = q.shape[0], q.device, q.dtype
    if out is None:
        qo = torch.empty(q.shape, dtype=io, device=dev)
        ko = None if k is None else torch.empty(k.shape, dtype=io, device=dev)
    else:
        qo, ko = out
        _check_all(dev, (qo, "out[0]", q.shape, io), (ko, "out[1]", q.shape if k is None else k.shape, io))
        if qo is None or (ko is None) != (k is None):
            raise ValueError("out must hold a tensor for q, and one for k where k is given")
    rc = lib().qknorm_step(q.data_ptr(), _ptr(k), q_weight.data_ptr(), _ptr(k_weight), _ptr(positions), _ptr(inv_freq), qo.data_ptr(),
                           _ptr(ko), batch, qh, kh, width, rotated, q.stride(0), 0 if k is None else k.stride(0), eps, dtype,
                           _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "qknorm_step")
    return qo, ko


def state_move(cache, src, dst, *, layers: bool = False, stream=None):
    """Copy, fork, compact and free rows of a cache in place: row ``dst[i]`` of
    ``cache`` [rows, ...] (or of every layer of [layers, rows, ...] with ``layers``)
    becomes what row ``src[i]`` held before the call, or zeros where ``src[i]`` is
    negative.  src and dst [moves] int32; rows may be the source of several moves and
    the target of another; targets are distinct, a negative one skips its move.  Any
    dtype.  Returns the cache."""
    at = 1 if layers else 0
    if cache.dim() <= at:
        raise ValueError(f"cache must have at least {at + 1} dimensions")
    if not cache.is_cuda:
        raise ValueError("state_move runs on CUDA tensors only")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    if src.dim() != 1 or src.shape[0] > STATE_MOVE_MAX:
        raise ValueError(f"src must be [0 to {STATE_MOVE_MAX}]")
    moves, rows = src.shape[0], cache.shape[at]
    _check_all(cache.device, (src, "src", (moves,), _I32), (dst, "dst", (moves,), _I32))
    _on_current(cache.device, "state_move")
    count = cache.shape[0] if layers else 1
    size = cache.numel() // (count * rows) * cache.element_size() if count * rows else 0
    rc = lib().state_move(cache.data_ptr(), src.data_ptr(), dst.data_ptr(), moves, count, rows, size, _stream_handle(stream))
    if rc != SSCAN_OK:
        raise SscanError(rc, "state_move")
    return cache


__all__ = ["sscan_fwd", "sscan_bwd", "sscan_step", "sscan_prompt", "pscan",
           "sconv_fwd", "sconv_bwd", "sconv_prompt", "sconv_step",
           "addnorm_fwd", "addnorm_bwd", "gatenorm_fwd", "gatenorm_bwd", "gatenorm_step",
           "lattn_fwd", "lattn_bwd", "lattn_prompt", "lattn_step",
           "qknorm_fwd", "qknorm_bwd", "qknorm_step", "state_move",
           "status_string", "get_last_error", "max_dstate",
           "last_launch_count", "last_plan", "load_library", "SscanError",
           "SIGNATURES", "LIB_PATH"]

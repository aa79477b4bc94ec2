"""Python binding of the state-space mixer's operators (include/wkv7_ssm.h):
argument marshalling only, as in wkv7.py.

    conv_forward / conv_step / conv_backward       short causal convolution
    ssm_forward / ssm_forward_train / ssm_step / ssm_backward   selective scan
    rmsnorm_forward / rmsnorm_backward             RMS norm with the residual's addition
    act8_save / act8_load                          8-bit activations

Per-token tensors are [B, T, D] (bf16 or fp32) and may be views with any token
and sequence stride as long as a token's channels are contiguous; parameters
and states are contiguous fp32.  All tensors of a call are on one device, which
need not be the current one; the call runs on ``stream`` (default: the device's
current stream), and what it allocates belongs to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional, Union

import torch

from . import wkv7
from .wkv7 import BF16, F32

E4M3 = 2
ACT8_BLOCK = 128
CODE_DTYPE = torch.float8_e4m3fn

EXPORTED_SYMBOLS = (
    "wkv7_act8_save", "wkv7_act8_load", "wkv7_rmsnorm_forward", "wkv7_rmsnorm_backward_workspace_size",
    "wkv7_rmsnorm_backward", "wkv7_conv_forward", "wkv7_conv_step", "wkv7_conv_backward_workspace_size",
    "wkv7_conv_backward", "wkv7_ssm_forward_workspace_size", "wkv7_ssm_saved_states_size", "wkv7_ssm_forward",
    "wkv7_ssm_step", "wkv7_ssm_backward_workspace_size", "wkv7_ssm_backward",
)

_CODE = {torch.float32: F32, torch.bfloat16: BF16}
_lib = None


class Act8(NamedTuple):
    """An activation [..., D] kept in 8 bits: e4m3 ``codes`` [..., D] and fp32
    ``scales`` [..., ceil(D / 128)], a power of two for each block of 128 channels."""
    codes: torch.Tensor
    scales: torch.Tensor


class NormOut(NamedTuple):
    y: Union[torch.Tensor, Act8]
    residual: Optional[torch.Tensor]
    rstd: torch.Tensor
    saved: Optional[Act8]


def load_library() -> ctypes.CDLL:
    """wkv7.load_library, with these operators' C signatures declared."""
    global _lib
    if _lib is not None:
        return _lib
    lib = wkv7.load_library()
    i, q, z, vp, f = ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float

    def sig(name, *args, res=i):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = list(args), res

    sig("wkv7_act8_save", q, i, i, vp, q, vp, vp, vp)
    sig("wkv7_act8_load", q, i, vp, vp, i, vp, vp)
    sig("wkv7_rmsnorm_forward", q, i, i, i, i, vp, q, vp, vp, f, vp, vp, vp, vp, vp, vp, vp)
    sig("wkv7_rmsnorm_backward_workspace_size", q, i, res=z)
    sig("wkv7_rmsnorm_backward", q, i, i, i, i, *[vp] * 9, z, vp)
    sig("wkv7_conv_forward", i, i, i, i, i, i, vp, q, q, vp, vp, vp, vp, vp, i, vp, vp, vp, vp, vp)
    sig("wkv7_conv_step", i, i, i, i, i, vp, q, vp, vp, vp, i, vp, vp)
    sig("wkv7_conv_backward_workspace_size", i, i, i, i, res=z)
    sig("wkv7_conv_backward", i, i, i, i, i, i, i, vp, q, q, vp, vp, vp, vp, vp, vp, i, vp, vp, vp, vp, vp, z, vp)
    sig("wkv7_ssm_forward_workspace_size", i, i, i, i, i, res=z)
    sig("wkv7_ssm_saved_states_size", i, i, i, i, res=z)
    scan = [vp, q, q, vp, q, q, vp, vp, q, q, vp, q, q, vp, vp, q, q, vp, vp, i]
    sig("wkv7_ssm_forward", *[i] * 7, *scan, vp, vp, vp, vp, vp, z, vp)
    sig("wkv7_ssm_step", *[i] * 6, vp, q, vp, q, vp, vp, q, vp, q, vp, vp, q, vp, vp, i, vp, vp)
    sig("wkv7_ssm_backward_workspace_size", *[i] * 6, res=z)
    sig("wkv7_ssm_backward", *[i] * 7, *scan, *[vp] * 12, vp, z, vp)
    _lib = lib
    return lib


# ---- arguments ------------------------------------------------------------------

def _code(t: torch.Tensor) -> int:
    c = _CODE.get(t.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return c


def _out_dtype(dtype, default: torch.dtype) -> torch.dtype:
    dtype = default if dtype is None else dtype
    if dtype not in _CODE:
        raise TypeError(f"unsupported dtype {dtype}")
    return dtype


def _y_dtype(y, y_dtype):
    """A given y's dtype is the call's; y_dtype beside it has to agree."""
    if y_dtype is not None and y.dtype != y_dtype:
        raise ValueError("y and y_dtype differ")


@contextlib.contextmanager
def _entered(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


_here = contextlib.nullcontext()


def _on(t: torch.Tensor, stream):
    """Context in which a call on ``t``'s device allocates and launches."""
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if stream is None and t.get_device() == torch.cuda.current_device():
        return _here
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {t.device}")
    return _entered(t.device, stream)


def _raw(t: torch.Tensor) -> int:
    """The current stream of ``t``'s (now current) device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _full(t, shape, dtype, dev, name):
    """Pointer of a contiguous tensor of that shape and type (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if t.get_device() != dev.index or not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous and on {dev}")
    return t.data_ptr()


def _tokens(t, shape, dtype, dev, name, inner=1):
    """Pointer and strides of a per-token input, whose last ``inner`` dimensions are contiguous."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    st = t.stride()
    if t.get_device() != dev.index or (st[-1] != 1 and shape[-1] > 1) or (inner == 2 and st[-2] != shape[-1] and shape[-2] > 1):
        raise ValueError(f"{name}: a token's channels must be contiguous, on {dev}")
    return (t.data_ptr(), *st[:-inner])


def _like(x, dtype):
    """An uninitialised tensor of x's shape on its device."""
    if dtype is x.dtype and x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(x.shape, dtype=dtype, device=x.device)


def _rows(t: torch.Tensor, name: str):
    """(rows, stride between rows) of a [..., D] tensor whose rows are evenly spaced."""
    D = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // D if D else 0), D
    if D > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: a row's channels must be contiguous")
    rows, ld, reach = 1, D, None
    for d in range(t.dim() - 2, -1, -1):
        n, s = t.shape[d], t.stride(d)
        if n == 1:
            continue
        if reach is None:
            ld = s
        elif s != reach:
            raise ValueError(f"{name}: rows must be evenly spaced")
        rows, reach = rows * n, s * n
    return (t.numel() // D if D else 0), ld


def _blocks(D: int) -> int:
    return (D + ACT8_BLOCK - 1) // ACT8_BLOCK


def _new_act8(shape, dev) -> Act8:
    return Act8(torch.empty(shape, dtype=CODE_DTYPE, device=dev),
                torch.empty((*shape[:-1], _blocks(shape[-1])), dtype=torch.float32, device=dev))


def _act8_ptrs(a, shape, dev, name):
    if a is None:
        return None, None
    return (_full(a.codes, shape, CODE_DTYPE, dev, name + ".codes"),
            _full(a.scales, (*shape[:-1], _blocks(shape[-1])), torch.float32, dev, name + ".scales"))


def _workspace(ws, nbytes, dev):
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    if ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"workspace: must be a contiguous uint8 tensor on {dev}")
    return ws


def _ws_args(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel())


def _done(fn, status, stream):
    if status != wkv7.OK or wkv7._status_checks:
        wkv7._check(fn, status, stream)


# ---- 8-bit activations ----------------------------------------------------------

def act8_save(x, *, out: Optional[Act8] = None, stream=None) -> Act8:
    """x [..., D] in 8 bits (include/wkv7_ssm.h has the format)."""
    lib = load_library()
    dt = _code(x)
    rows, ld = _rows(x, "x")
    with _on(x, stream):
        if out is None:
            out = _new_act8(x.shape, x.device)
            c, s = out.codes.data_ptr(), out.scales.data_ptr()
        else:
            c, s = _act8_ptrs(out, x.shape, x.device, "out")
        st = lib.wkv7_act8_save(rows, x.shape[-1], dt, x.data_ptr(), ld, c, s, _raw(x))
        _done("wkv7_act8_save", st, stream)
    return out


def act8_load(a: Act8, dtype=torch.bfloat16, *, out=None, stream=None):
    """The values [..., D] that 8-bit codes stand for (exact in bf16 and fp32)."""
    lib = load_library()
    dtype = _out_dtype(dtype, torch.bfloat16)
    shape, dev = a.codes.shape, a.codes.device
    with _on(a.codes, stream):
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
            op = out.data_ptr()
        else:
            op = _full(out, shape, dtype, dev, "out")
        c, s = _act8_ptrs(a, shape, dev, "a")
        D = shape[-1]
        st = lib.wkv7_act8_load(a.codes.numel() // D if D else 0, D, c, s, _CODE[dtype], op, _raw(out))
        _done("wkv7_act8_load", st, stream)
    return out


# ---- RMS norm -------------------------------------------------------------------

def rmsnorm_forward(x, weight, residual=None, *, eps=1e-6, out8=False, save8=False, y=None, y_dtype=None,
                    residual_out=None, saved: Optional[Act8] = None, stream=None) -> NormOut:
    """s = x + residual;  y = weight s / sqrt(mean(s^2) + eps) over the last dimension.

    x [..., D], residual the same shape (its own dtype), weight [D] fp32.
    ``out8`` gives y as an Act8, else it is of ``y_dtype`` (x's).  ``save8`` also
    keeps s as an Act8 for ``rmsnorm_backward``.  The result's ``residual`` is s
    in the residual's dtype (None without a residual; ``residual_out`` may be
    ``residual`` itself), ``rstd`` [...] fp32."""
    lib = load_library()
    dev, shape = x.device, x.shape
    D = shape[-1]
    rows, ld = _rows(x, "x")
    xc = _code(x)
    rc = xc if residual is None else _code(residual)
    if out8 and y_dtype is not None:
        raise ValueError("y_dtype: not with out8")
    if y is not None and out8 != isinstance(y, Act8):
        raise ValueError("y: an Act8 with out8, a tensor without")
    with _on(x, stream):
        if out8:
            yc = E4M3
            if y is None:
                y = _new_act8(shape, dev)
                yp, ysp = y.codes.data_ptr(), y.scales.data_ptr()
            else:
                yp, ysp = _act8_ptrs(y, shape, dev, "y")
        else:
            if y is None:
                y = _like(x, _out_dtype(y_dtype, x.dtype))
            else:
                _y_dtype(y, y_dtype)
            yc, yp, ysp = _code(y), _full(y, shape, y.dtype, dev, "y"), None
        if residual is not None and residual_out is None:
            residual_out = torch.empty_like(residual)
        if residual is None and residual_out is not None:
            raise ValueError("residual_out: only with a residual")
        if save8 and saved is None:
            saved = _new_act8(shape, dev)
        sc, ss = _act8_ptrs(saved, shape, dev, "saved")
        rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        rdt = None if residual is None else residual.dtype
        st = lib.wkv7_rmsnorm_forward(rows, D, xc, rc, yc, x.data_ptr(), ld, _full(residual, shape, rdt, dev, "residual"),
                                      _full(weight, (D,), torch.float32, dev, "weight"), eps,
                                      _full(residual_out, shape, rdt, dev, "residual_out"), yp, ysp, sc, ss,
                                      rstd.data_ptr(), _raw(x))
        _done("wkv7_rmsnorm_forward", st, stream)
    return NormOut(y, residual_out, rstd, saved)


def rmsnorm_backward_workspace_size(rows, D) -> int:
    return load_library().wkv7_rmsnorm_backward_workspace_size(rows, D)


def rmsnorm_backward(dy, s: Union[torch.Tensor, Act8], rstd, weight, *, dresidual=None, grad_dtype=torch.float32,
                     dx=None, workspace=None, stream=None):
    """(dx, dweight): gradients of x (the residual's is the same) and weight.
    ``s`` is the normalised sum: the forward's ``saved``, its ``residual``, or x."""
    lib = load_library()
    dev, shape, D = dy.device, tuple(dy.shape), dy.shape[-1]
    rows = dy.numel() // D if D else 0
    gd = _out_dtype(grad_dtype, torch.float32)
    with _on(dy, stream):
        if isinstance(s, Act8):
            sc, (sp, ssp) = E4M3, _act8_ptrs(s, shape, dev, "s")
        else:
            sc, sp, ssp = _code(s), _full(s, shape, s.dtype, dev, "s"), None
        if dx is None:
            dx = torch.empty(shape, dtype=gd, device=dev)
        dweight = torch.empty(D, dtype=torch.float32, device=dev)
        ws = _workspace(workspace, lib.wkv7_rmsnorm_backward_workspace_size(rows, D), dev)
        st = lib.wkv7_rmsnorm_backward(rows, D, sc, _code(dy), _CODE[gd], sp, ssp,
                                       _full(rstd, shape[:-1], torch.float32, dev, "rstd"),
                                       _full(weight, (D,), torch.float32, dev, "weight"),
                                       _full(dy, shape, dy.dtype, dev, "dy"),
                                       _full(dresidual, shape, gd, dev, "dresidual"),
                                       _full(dx, shape, gd, dev, "dx"), dweight.data_ptr(), *_ws_args(ws), _raw(dy))
        _done("wkv7_rmsnorm_backward", st, stream)
    return dx, dweight


# ---- short causal convolution ------------------------------------------------------

def _conv_x(x, dev, y_dtype, shape):
    """(code, pointer, strides, scales pointer, the state's dtype) of a tensor or an Act8."""
    if isinstance(x, Act8):
        c, s = _act8_ptrs(x, shape, dev, "x")
        return E4M3, (c, 0, 0), s, y_dtype
    return _code(x), _tokens(x, shape, x.dtype, dev, "x"), None, x.dtype


def conv_forward(x: Union[torch.Tensor, Act8], weight, bias=None, state=None, *, silu=True, lens=None, y=None,
                 y_dtype=None, state_out=None, return_state=False, save8=False, saved: Optional[Act8] = None,
                 stream=None):
    """y [B, T, D] of the causal convolution of x with weight [D, W] (fp32, W = 2,
    3 or 4), bias [D] fp32, after ``state`` [B, W - 1, D] (the inputs before the
    first token; None = zeros).  ``lens`` [B] int32 ends sequences early: rows of
    y behind a sequence's end stay as they are (unset in a y that is allocated here).

    Returns y, or a tuple (y, state_out, saved) of what was asked for:
    ``return_state`` adds the last W - 1 inputs, ``save8`` x as an Act8.  With an
    Act8 for x (its recomputation in a backward pass) y is of ``y_dtype``, bf16
    unless given."""
    lib = load_library()
    first = x.codes if isinstance(x, Act8) else x
    dev, shape = first.device, tuple(first.shape)
    B, T, D = shape
    W = weight.shape[-1]
    with _on(first, stream):
        if y is None:
            y = torch.empty(shape, dtype=_out_dtype(y_dtype, torch.bfloat16 if isinstance(x, Act8) else x.dtype),
                            device=dev)
        else:
            _y_dtype(y, y_dtype)
        xc, (xp, xb, xt), xs, sdt = _conv_x(x, dev, y.dtype, shape)
        if return_state and state_out is None:
            state_out = torch.empty((B, W - 1, D), dtype=sdt, device=dev)
        if save8 and saved is None:
            saved = _new_act8(shape, dev)
        qc, qs = _act8_ptrs(saved, shape, dev, "saved")
        st = lib.wkv7_conv_forward(B, T, D, W, xc, _code(y), xp, xb, xt, xs,
                                   _full(weight, (D, W), torch.float32, dev, "weight"),
                                   _full(bias, (D,), torch.float32, dev, "bias"),
                                   _full(state, (B, W - 1, D), sdt, dev, "state"),
                                   _full(lens, (B,), torch.int32, dev, "lens"), int(silu),
                                   _full(y, shape, y.dtype, dev, "y"),
                                   _full(state_out, (B, W - 1, D), sdt, dev, "state_out"), qc, qs, _raw(first))
        _done("wkv7_conv_forward", st, stream)
    extra = tuple(v for v in (state_out, saved) if v is not None)
    return (y,) + extra if extra else y


def conv_step(x, weight, bias, state, *, silu=True, y=None, y_dtype=None, stream=None):
    """One token x [B, D]; ``state`` [B, W - 1, D] of x's dtype moves on in place."""
    lib = load_library()
    dev = x.device
    B, D = x.shape
    W = weight.shape[-1]
    xp, xb = _tokens(x, (B, D), x.dtype, dev, "x")
    with _on(x, stream):
        if y is None:
            y = _like(x, _out_dtype(y_dtype, x.dtype))
            yp = y.data_ptr()
        else:
            _y_dtype(y, y_dtype)
            yp = _full(y, (B, D), y.dtype, dev, "y")
        st = lib.wkv7_conv_step(B, D, W, _code(x), _code(y), xp, xb, _full(weight, (D, W), torch.float32, dev, "weight"),
                                _full(bias, (D,), torch.float32, dev, "bias"),
                                _full(state, (B, W - 1, D), x.dtype, dev, "state"), silu, yp, _raw(x))
        _done("wkv7_conv_step", st, stream)
    return y


def conv_backward_workspace_size(B, T, D, W) -> int:
    return load_library().wkv7_conv_backward_workspace_size(B, T, D, W)


def conv_backward(x: Union[torch.Tensor, Act8], weight, bias, dy, state=None, dstate_out=None, *, silu=True,
                  grad_dtype=torch.float32, dx=None, workspace=None, stream=None):
    """(dx, dweight, dbias, dstate) of L = sum(dy y) + sum(dstate_out state_out);
    dbias and dstate are None where the forward had no bias or state.  ``x`` may
    be its Act8 (``state`` is then of grad_dtype)."""
    lib = load_library()
    dev, shape = dy.device, tuple(dy.shape)
    B, T, D = shape
    W = weight.shape[-1]
    gd = _out_dtype(grad_dtype, torch.float32)
    with _on(dy, stream):
        xc, (xp, xb, xt), xs, sdt = _conv_x(x, dev, gd, shape)
        if dx is None:
            dx = torch.empty(shape, dtype=gd, device=dev)
        dweight = torch.empty((D, W), dtype=torch.float32, device=dev)
        dbias = None if bias is None else torch.empty(D, dtype=torch.float32, device=dev)
        dstate = None if state is None else torch.empty((B, W - 1, D), dtype=torch.float32, device=dev)
        ws = _workspace(workspace, lib.wkv7_conv_backward_workspace_size(B, T, D, W), dev)
        st = lib.wkv7_conv_backward(B, T, D, W, xc, _code(dy), _CODE[gd], xp, xb, xt, xs,
                                    _full(weight, (D, W), torch.float32, dev, "weight"),
                                    _full(bias, (D,), torch.float32, dev, "bias"),
                                    _full(state, (B, W - 1, D), sdt, dev, "state"), _full(dy, shape, dy.dtype, dev, "dy"),
                                    _full(dstate_out, (B, W - 1, D), torch.float32, dev, "dstate_out"), int(silu),
                                    _full(dx, shape, gd, dev, "dx"), dweight.data_ptr(),
                                    None if dbias is None else dbias.data_ptr(),
                                    None if dstate is None else dstate.data_ptr(), *_ws_args(ws), _raw(dy))
        _done("wkv7_conv_backward", st, stream)
    return dx, dweight, dbias, dstate


# ---- selective scan ----------------------------------------------------------------

def _scan_args(u, delta, A, B, C, D, z, dt_bias):
    """Sizes and the C call's shared arguments (pointers and strides), for sequences or single tokens."""
    dev, dt = u.device, u.dtype
    lead = tuple(u.shape[:-1])
    Dn, N, G = u.shape[-1], A.shape[-1], B.shape[-2]
    bc = lead + (G, N)
    none = (None,) + (0,) * len(lead)
    args = (*_tokens(u, lead + (Dn,), dt, dev, "u"), *_tokens(delta, lead + (Dn,), dt, dev, "delta"),
            _full(A, (Dn, N), torch.float32, dev, "A"), *_tokens(B, bc, dt, dev, "B", 2), *_tokens(C, bc, dt, dev, "C", 2),
            _full(D, (Dn,), torch.float32, dev, "D"),
            *(none if z is None else _tokens(z, lead + (Dn,), dt, dev, "z")),
            _full(dt_bias, (Dn,), torch.float32, dev, "dt_bias"))
    return Dn, N, G, args


def ssm_forward_workspace_size(B, T, D, N, G=1) -> int:
    return load_library().wkv7_ssm_forward_workspace_size(B, T, D, N, G)


def ssm_saved_states_size(B, T, D, N) -> int:
    return load_library().wkv7_ssm_saved_states_size(B, T, D, N)


def _forward(u, delta, A, B, C, D, z, dt_bias, state0, softplus, lens, y, y_dtype, stateT, states, workspace,
             return_state, stream):
    lib = load_library()
    dev = u.device
    Bn, T, _ = u.shape
    with _on(u, stream):
        Dn, N, G, args = _scan_args(u, delta, A, B, C, D, z, dt_bias)
        if y is None:
            y = _like(u, _out_dtype(y_dtype, u.dtype))
        else:
            _y_dtype(y, y_dtype)
        if return_state and stateT is None:
            stateT = torch.empty((Bn, Dn, N), dtype=torch.float32, device=dev)
        if states is True:
            states = torch.empty((Bn, (T + 15) // 16, Dn, N), dtype=torch.float32, device=dev)
        ws = _workspace(workspace, lib.wkv7_ssm_forward_workspace_size(Bn, T, Dn, N, G), dev)
        sh = (Bn, Dn, N)
        st = lib.wkv7_ssm_forward(Bn, T, Dn, N, G, _code(u), _code(y), *args,
                                  _full(state0, sh, torch.float32, dev, "state0"), int(softplus),
                                  _full(lens, (Bn,), torch.int32, dev, "lens"), _full(y, (Bn, T, Dn), y.dtype, dev, "y"),
                                  _full(stateT, sh, torch.float32, dev, "stateT"),
                                  _full(states, (Bn, (T + 15) // 16, Dn, N), torch.float32, dev, "states"),
                                  *_ws_args(ws), _raw(u))
        _done("wkv7_ssm_forward", st, stream)
    return y, stateT, states


def ssm_forward(u, delta, A, B, C, D=None, z=None, dt_bias=None, state0=None, *, softplus=True, lens=None, y=None,
                y_dtype=None, stateT=None, workspace=None, return_state=True, stream=None):
    """(y [B,T,D], stateT [B,D,N]) of the selective scan

        dt = softplus(delta + dt_bias),  h_t = exp(dt A) h_{t-1} + dt u_t B_t,
        y_t = (C_t . h_t + D u_t) z_t sigmoid(z_t)

    u, delta, z [B, T, D] and B, C [B, T, G, N] of one dtype; A [D, N], D and
    dt_bias [D], state0 [B, D, N] fp32 (None = zeros; z None = no gate); N <= 64.
    ``lens`` [B] int32 ends sequences early: rows of y behind a sequence's end
    stay as they are (unset in a y that is allocated here), and stateT is the state
    at its end."""
    y, stateT, _ = _forward(u, delta, A, B, C, D, z, dt_bias, state0, softplus, lens, y, y_dtype, stateT, None, workspace,
                            return_state, stream)
    return (y, stateT) if return_state else y


def ssm_forward_train(u, delta, A, B, C, D=None, z=None, dt_bias=None, state0=None, *, softplus=True, y=None,
                      y_dtype=None, stateT=None, states=None, workspace=None, stream=None):
    """(y, stateT, states): ``ssm_forward`` that keeps the state before every 16th
    token, [B, ceil(T / 16), D, N] fp32, for ``ssm_backward``."""
    return _forward(u, delta, A, B, C, D, z, dt_bias, state0, softplus, None, y, y_dtype, stateT,
                    True if states is None else states, workspace, True, stream)


def ssm_step(u, delta, A, B, C, state, D=None, z=None, dt_bias=None, *, softplus=True, y=None, y_dtype=None,
             stream=None):
    """One token: u, delta, z [B, D] and B, C [B, G, N]; the fp32 state [B, D, N] is updated in place."""
    lib = load_library()
    dev = u.device
    Bn = u.shape[0]
    with _on(u, stream):
        Dn, N, G, args = _scan_args(u, delta, A, B, C, D, z, dt_bias)
        if y is None:
            y = _like(u, _out_dtype(y_dtype, u.dtype))
            yp = y.data_ptr()
        else:
            _y_dtype(y, y_dtype)
            yp = _full(y, (Bn, Dn), y.dtype, dev, "y")
        st = lib.wkv7_ssm_step(Bn, Dn, N, G, _code(u), _code(y), *args,
                               _full(state, (Bn, Dn, N), torch.float32, dev, "state"), softplus, yp, _raw(u))
        _done("wkv7_ssm_step", st, stream)
    return y


def ssm_backward_workspace_size(B, T, D, N, G=1, with_states=True) -> int:
    return load_library().wkv7_ssm_backward_workspace_size(B, T, D, N, G, int(with_states))


class SsmGrads(NamedTuple):
    u: torch.Tensor
    delta: torch.Tensor
    A: torch.Tensor
    B: torch.Tensor
    C: torch.Tensor
    D: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    dt_bias: Optional[torch.Tensor]
    state0: torch.Tensor


def ssm_backward(u, delta, A, B, C, dy, D=None, z=None, dt_bias=None, state0=None, dstateT=None, *, softplus=True,
                 states=None, grad_dtype=torch.float32, workspace=None, stream=None) -> SsmGrads:
    """Gradients of L = sum(dy y) + sum(dstateT stateT) with respect to every
    input: per-token ones in ``grad_dtype``, parameters and state0 in fp32.
    ``states``: what ``ssm_forward_train`` kept (None computes them from state0)."""
    lib = load_library()
    dev = u.device
    Bn, T, _ = u.shape
    gd = _out_dtype(grad_dtype, torch.float32)
    with _on(u, stream):
        Dn, N, G, args = _scan_args(u, delta, A, B, C, D, z, dt_bias)

        def new(*shape, dtype=gd):
            return torch.empty(shape, dtype=dtype, device=dev)

        f32 = torch.float32
        g = SsmGrads(new(Bn, T, Dn), new(Bn, T, Dn), new(Dn, N, dtype=f32), new(Bn, T, G, N), new(Bn, T, G, N),
                     None if D is None else new(Dn, dtype=f32), None if z is None else new(Bn, T, Dn),
                     None if dt_bias is None else new(Dn, dtype=f32), new(Bn, Dn, N, dtype=f32))
        ws = _workspace(workspace, lib.wkv7_ssm_backward_workspace_size(Bn, T, Dn, N, G, int(states is not None)), dev)
        sh = (Bn, Dn, N)
        st = lib.wkv7_ssm_backward(Bn, T, Dn, N, G, _code(u), _CODE[gd], *args,
                                   _full(state0, sh, f32, dev, "state0"), int(softplus),
                                   _full(states, (Bn, (T + 15) // 16, Dn, N), f32, dev, "states"),
                                   _full(dy, (Bn, T, Dn), u.dtype, dev, "dy"), _full(dstateT, sh, f32, dev, "dstateT"),
                                   g.u.data_ptr(), g.delta.data_ptr(), g.A.data_ptr(), g.B.data_ptr(), g.C.data_ptr(),
                                   None if D is None else g.D.data_ptr(), None if z is None else g.z.data_ptr(),
                                   None if dt_bias is None else g.dt_bias.data_ptr(), g.state0.data_ptr(), *_ws_args(ws),
                                   _raw(u))
        _done("wkv7_ssm_backward", st, stream)
    return g

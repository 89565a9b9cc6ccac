"""Thin Python binding of libetp's dense operators (include/etp_dense.h), same
names as the C ABI: the linear layer and the layer norm of the radial and node
networks with their VJPs, and the orthogonalised update of weight matrices.

As in ``etp``: argument marshalling only, torch's current HIP stream unless
given, ``EtpError`` for every non-zero status. Feature matrices are 2-D tensors
(float32 or bfloat16, all of one call alike) whose rows may be strided
(``stride(1) == 1``); bias, gamma, beta, row statistics and weight gradients are
float32.
"""
from __future__ import annotations

import ctypes

import torch

from .etp import (ETP_BF16, ETP_F32, ETP_FLAG_ACCUMULATE, EtpError, _check, lib)  # noqa: F401
from .etp import _stream as _any_stream

ETP_ACT_NONE, ETP_ACT_SILU, ETP_ACT_GELU = 0, 1, 2

# every symbol include/etp_dense.h declares
ABI_SYMBOLS = ("etp_linear", "etp_linear_vjp", "etp_linear_vjp_workspace", "etp_layer_norm", "etp_layer_norm_vjp",
               "etp_layer_norm_vjp_workspace", "etp_orthogonalize", "etp_orthogonalize_workspace")


def _declare():
    vp, st, i32, i64, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32
    f32, sz, psz = ctypes.c_float, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "etp_linear": [i64, i32, i32, i32, vp, i64, vp, vp, i32, vp, i64, vp, i64, vp, i64, vp],
        "etp_linear_vjp": [i64, i32, i32, i32, vp, i64, vp, vp, i64, i32, vp, i64, vp, i64, vp, vp, u32, vp, sz, vp],
        "etp_linear_vjp_workspace": [i64, i32, i32, i32, psz],
        "etp_layer_norm": [i64, i32, i32, vp, i64, vp, vp, f32, vp, i64, vp, vp, vp],
        "etp_layer_norm_vjp": [i64, i32, i32, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, u32, vp, sz, vp],
        "etp_layer_norm_vjp_workspace": [i64, i32, i32, psz],
        "etp_orthogonalize": [i32, i32, i32, i32, vp, i32, vp, f32, vp, vp, sz, vp],
        "etp_orthogonalize_workspace": [i32, i32, i32, i32, psz],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = st, args


_declare()

_CODE = {torch.float32: ETP_F32, torch.bfloat16: ETP_BF16}


def _code(dtype) -> int:
    if dtype not in _CODE:
        raise ValueError(f"features must be torch.float32 or torch.bfloat16, got {dtype}")
    return _CODE[dtype]


# torch's current stream of a device as a plain handle: the stream object that
# torch.cuda.current_stream builds takes longer than all the other marshalling
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, x):
    if stream is None and _raw_stream is not None:
        return _raw_stream(x.get_device())
    return _any_stream(stream)


def _rows(t, name, dtype, rows, cols, optional=False):
    """(device pointer, row pitch) of a [rows][cols] tensor with unit column stride."""
    if t is None:
        if optional:
            return None, 0
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}][{cols}], got {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    pitch, unit = t.stride()
    if rows < 2:
        pitch = cols
    if cols > 1 and unit != 1 or pitch < cols:
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap, got strides {t.stride()}")
    return t.data_ptr(), pitch


def _dense(t, name, dtype, numel, optional=False):
    """Device pointer of a contiguous tensor of numel elements (None -> NULL if optional)."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and have {numel} elements, got {list(t.shape)}, strides {t.stride()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.data_ptr()


def _dense_matrix(t, name, dtype, rows, cols, n_mats=1, optional=False):
    """_dense of [rows][cols] matrices back to back: flat, or with that shape in the last two dimensions."""
    if t is not None and t.dim() > 1 and t.shape[-2:] != (rows, cols):
        raise ValueError(f"{name} must be [{rows}][{cols}], got {list(t.shape)}")
    return _dense(t, name, dtype, n_mats * rows * cols, optional)


def _workspace(ws):
    return (None, 0) if ws is None else (_dense(ws, "ws", ws.dtype, ws.numel()), ws.numel() * ws.element_size())


def _bytes(name, *args) -> int:
    b = ctypes.c_size_t()
    _check(getattr(lib, name)(*args, ctypes.byref(b)), name)
    return b.value


def _matrix(x, name):
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {list(x.shape)}")
    return x.shape


def etp_linear(x, W, y, bias=None, activation: int = ETP_ACT_NONE, residual=None, z=None, stream=None):
    """z = x @ W + bias, y = act(z) + residual. x [M, K], W [K, N]; residual, y, z [M, N]; bias float [N]. z (what
    the VJP of a layer with an activation needs) is written when given."""
    M, K = _matrix(x, "x")
    N, dt = W.shape[-1], x.dtype
    code = _code(dt)
    xp, ldx = _rows(x, "x", dt, M, K)
    rp, ldr = _rows(residual, "residual", dt, M, N, True)
    yp, ldy = _rows(y, "y", dt, M, N)
    zp, ldz = _rows(z, "z", dt, M, N, True)
    _check(lib.etp_linear(M, K, N, code, xp, ldx, _dense_matrix(W, "W", dt, K, N),
                          _dense(bias, "bias", torch.float32, N, True), activation, rp, ldr, yp, ldy, zp, ldz,
                          _stream(stream, x)), "etp_linear")


def etp_linear_vjp_workspace(n_rows: int, n_in: int, n_out: int, dtype=torch.float32) -> int:
    return _bytes("etp_linear_vjp_workspace", n_rows, n_in, n_out, _code(dtype))


def etp_linear_vjp(x, W, grad_y, z=None, activation: int = ETP_ACT_NONE, grad_x=None, grad_W=None, grad_b=None,
                   ws=None, flags: int = 0, stream=None):
    """VJP of etp_linear: grad_x [M, K], grad_W float [K, N], grad_b float [N] (each optional; x may be None without
    grad_W, W without grad_x); ws: etp_linear_vjp_workspace(M, K, N, dtype) bytes."""
    M, N = _matrix(grad_y, "grad_y")
    dt = grad_y.dtype
    if W is not None:
        K = W.shape[0]
    else:
        given = x if x is not None else grad_x
        K = 1 if given is None else _matrix(given, "x" if x is not None else "grad_x")[1]  # (grad_b has no K)
    code = _code(dt)
    Wp = _dense_matrix(W, "W", dt, K, N, optional=True)
    xp, ldx = _rows(x, "x", dt, M, K, True)
    zp, ldz = _rows(z, "z", dt, M, N, True)
    gp, ldg = _rows(grad_y, "grad_y", dt, M, N)
    op, ldo = _rows(grad_x, "grad_x", dt, M, K, True)
    wp, wb = _workspace(ws)
    f32 = torch.float32
    _check(lib.etp_linear_vjp(M, K, N, code, xp, ldx, Wp, zp, ldz, activation, gp, ldg, op, ldo,
                              _dense_matrix(grad_W, "grad_W", f32, K, N, optional=True),
                              _dense(grad_b, "grad_b", f32, N, True), flags, wp, wb, _stream(stream, grad_y)),
           "etp_linear_vjp")


def etp_layer_norm(x, y, gamma=None, beta=None, eps: float = 1e-5, mean=None, rstd=None, stream=None):
    """y = (x - mean) * rstd * gamma + beta over each row of x [M, C]; mean, rstd float [M] are written when given
    (the VJP needs both)."""
    M, C = _matrix(x, "x")
    dt, f32 = x.dtype, torch.float32
    code = _code(dt)
    xp, ldx = _rows(x, "x", dt, M, C)
    yp, ldy = _rows(y, "y", dt, M, C)
    _check(lib.etp_layer_norm(M, C, code, xp, ldx, _dense(gamma, "gamma", f32, C, True),
                              _dense(beta, "beta", f32, C, True), eps, yp, ldy,
                              _dense(mean, "mean", f32, M, True), _dense(rstd, "rstd", f32, M, True),
                              _stream(stream, x)), "etp_layer_norm")


def etp_layer_norm_vjp_workspace(n_rows: int, n_cols: int, dtype=torch.float32) -> int:
    return _bytes("etp_layer_norm_vjp_workspace", n_rows, n_cols, _code(dtype))


def etp_layer_norm_vjp(x, mean, rstd, grad_y, gamma=None, grad_x=None, grad_gamma=None, grad_beta=None, ws=None,
                       flags: int = 0, stream=None):
    """VJP of etp_layer_norm: grad_x [M, C], grad_gamma and grad_beta float [C] (each optional); ws:
    etp_layer_norm_vjp_workspace(M, C, dtype) bytes."""
    M, C = _matrix(x, "x")
    dt, f32 = x.dtype, torch.float32
    code = _code(dt)
    xp, ldx = _rows(x, "x", dt, M, C)
    gp, ldg = _rows(grad_y, "grad_y", dt, M, C)
    op, ldo = _rows(grad_x, "grad_x", dt, M, C, True)
    wp, wb = _workspace(ws)
    _check(lib.etp_layer_norm_vjp(M, C, code, xp, ldx, _dense(gamma, "gamma", f32, C, True),
                                  _dense(mean, "mean", f32, M), _dense(rstd, "rstd", f32, M), gp, ldg, op, ldo,
                                  _dense(grad_gamma, "grad_gamma", f32, C, True),
                                  _dense(grad_beta, "grad_beta", f32, C, True), flags, wp, wb,
                                  _stream(stream, x)), "etp_layer_norm_vjp")


def etp_orthogonalize_workspace(n_mats: int, rows: int, cols: int, dtype=torch.float32) -> int:
    return _bytes("etp_orthogonalize_workspace", n_mats, rows, cols, _code(dtype))


def etp_orthogonalize(G, X, steps: int = 5, coef=None, eps: float = 1e-7, ws=None, stream=None):
    """X = the Newton-Schulz orthogonalisation of each matrix of G [rows, cols] or [n_mats, rows, cols]; coef: three
    numbers or None (the defaults of the C ABI); ws: etp_orthogonalize_workspace(n_mats, rows, cols, dtype) bytes."""
    if G.dim() not in (2, 3):
        raise ValueError(f"G must be [rows][cols] or [n_mats][rows][cols], got {list(G.shape)}")
    n = G.shape[0] if G.dim() == 3 else 1
    dt = G.dtype
    code = _code(dt)
    r, k = G.shape[-2:]
    wp, wb = _workspace(ws)
    c = None if coef is None else (ctypes.c_float * 3)(*coef)
    _check(lib.etp_orthogonalize(n, r, k, code, _dense(G, "G", dt, G.numel()), steps, c, eps,
                                 _dense_matrix(X, "X", dt, r, k, n), wp, wb, _stream(stream, G)), "etp_orthogonalize")

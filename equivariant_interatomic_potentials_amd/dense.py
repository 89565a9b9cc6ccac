"""Thin Python binding of libetp's dense operators (include/etp_dense.h), same
names as the C ABI: the linear layer and the layer norm of the radial and node
networks with their VJPs, the linear layer with a matrix for each group of rows
(elements, pairs of elements) and the grouping of rows by type, the norm of all
gradients with clipping, and the orthogonalised update of weight matrices.

As in ``etp``: argument marshalling only, torch's current HIP stream unless
given, ``EtpError`` for every non-zero status. Feature matrices are 2-D tensors
(float32 or bfloat16, all of one call alike) whose rows may be strided
(``stride(1) == 1``); bias, gamma, beta, row statistics and weight gradients are
float32. The rows' groups are int32. The grouped layer and the gradient list also
check that their tensors share a device, and launch on that one whichever is current.
"""
from __future__ import annotations

import ctypes
import operator
import weakref

import numpy
import torch

from .etp import (ETP_BF16, ETP_F32, ETP_FLAG_ACCUMULATE, EtpError, _check, lib)  # noqa: F401
from .etp import _stream as _any_stream

ETP_ACT_NONE, ETP_ACT_SILU, ETP_ACT_GELU = 0, 1, 2

# every symbol include/etp_dense.h declares
ABI_SYMBOLS = ("etp_linear", "etp_linear_vjp", "etp_linear_vjp_workspace", "etp_layer_norm", "etp_layer_norm_vjp",
               "etp_layer_norm_vjp_workspace", "etp_orthogonalize", "etp_orthogonalize_workspace",
               "etp_group_rows", "etp_group_rows_workspace", "etp_grouped_linear", "etp_grouped_linear_vjp",
               "etp_grouped_linear_vjp_workspace", "etp_grad_norm", "etp_clip_grads", "etp_grad_norm_workspace")


class etp_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32)]


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
        "etp_group_rows": [i64, i32, vp, vp, vp, vp, sz, vp],
        "etp_group_rows_workspace": [i64, i32, psz],
        "etp_grouped_linear": [i64, i32, vp, vp, i32, i32, i32, vp, i64, vp, vp, i32, vp, i64, vp, i64, vp, i64, vp],
        "etp_grouped_linear_vjp": [i64, i32, vp, vp, i32, i32, i32, vp, i64, vp, vp, i64, i32, vp, i64, vp, i64, vp,
                                   vp, u32, vp, sz, vp],
        "etp_grouped_linear_vjp_workspace": [i64, i32, i32, i32, i32, psz],
        "etp_grad_norm": [i32, vp, vp, vp, sz, vp],
        "etp_clip_grads": [i32, vp, f32, vp, vp, vp, sz, vp],
        "etp_grad_norm_workspace": [i32, vp, psz],
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


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name, device, stream, args):
    """One call on the device (its number) its tensors live on: a stream belongs to a device, the launch to the current
    one."""
    f = getattr(lib, name)
    if _current_device() == device:
        st = f(*args, _stream_of(stream, device))
    else:
        with torch.cuda.device(device):
            st = f(*args, _stream_of(stream, device))
    if st:
        _check(st, name)


def _stream_of(stream, device):
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _any_stream(stream)


def _share_device(first, *tensors):
    """The number of the tensors' device."""
    device = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors of one call must share a device, got {first.device} and {t.device}")
    return device


def etp_group_rows_workspace(n_rows: int, n_groups: int) -> int:
    return _bytes("etp_group_rows_workspace", n_rows, n_groups)


def etp_group_rows(ids, group_ptr, order, ws=None, stream=None):
    """group_ptr [G + 1] and order [M], int32: the rows of ids int32 [M] by group, in row order within each, rows whose
    id is none of 0 .. G - 1 last; ws: etp_group_rows_workspace(M, G) bytes."""
    M, G, i32 = ids.numel(), group_ptr.numel() - 1, torch.int32
    wp, wb = _workspace(ws)
    args = (M, G, _dense(ids, "ids", i32, M), _dense(group_ptr, "group_ptr", i32, G + 1),
            _dense(order, "order", i32, M), wp, wb)
    _call("etp_group_rows", _share_device(ids, group_ptr, order, ws), stream, args)


def _groups(group_ptr, order, rows):
    """(number of groups, pointers of the offsets and of the order)"""
    G = group_ptr.numel() - 1
    return G, _dense(group_ptr, "group_ptr", torch.int32, G + 1), _dense(order, "order", torch.int32, rows, True)


def etp_grouped_linear(x, W, y, group_ptr, order=None, bias=None, activation: int = ETP_ACT_NONE, residual=None, z=None,
                       stream=None):
    """z = x @ W[g] + bias[g], y = act(z) + residual for the rows order[group_ptr[g]:group_ptr[g + 1]] of each group g
    (order None: the rows themselves). x [M, K], W [G, K, N]; residual, y, z [M, N]; bias float [G, N]. Rows in no group
    are left alone."""
    M, K = _matrix(x, "x")
    N, dt = W.shape[-1], x.dtype
    code = _code(dt)
    G, gp, op = _groups(group_ptr, order, M)
    xp, ldx = _rows(x, "x", dt, M, K)
    rp, ldr = _rows(residual, "residual", dt, M, N, True)
    yp, ldy = _rows(y, "y", dt, M, N)
    zp, ldz = _rows(z, "z", dt, M, N, True)
    args = (M, G, gp, op, K, N, code, xp, ldx, _dense_matrix(W, "W", dt, K, N, G),
            _dense(bias, "bias", torch.float32, G * N, True), activation, rp, ldr, yp, ldy, zp, ldz)
    _call("etp_grouped_linear", _share_device(x, W, y, group_ptr, order, bias, residual, z), stream, args)


def etp_grouped_linear_vjp_workspace(n_rows: int, n_groups: int, n_in: int, n_out: int, dtype=torch.float32) -> int:
    return _bytes("etp_grouped_linear_vjp_workspace", n_rows, n_groups, n_in, n_out, _code(dtype))


def etp_grouped_linear_vjp(x, W, grad_y, group_ptr, order=None, z=None, activation: int = ETP_ACT_NONE, grad_x=None,
                           grad_W=None, grad_b=None, ws=None, flags: int = 0, stream=None):
    """VJP of etp_grouped_linear: grad_x [M, K], grad_W float [G, K, N], grad_b float [G, N] (each optional; x may be
    None without grad_W, W without grad_x); ws: etp_grouped_linear_vjp_workspace(M, G, K, N, dtype) bytes."""
    M, N = _matrix(grad_y, "grad_y")
    dt = grad_y.dtype
    if W is not None:
        if W.dim() != 3:
            raise ValueError(f"W must be [groups][rows][cols], got {list(W.shape)}")
        K = W.shape[1]
    else:
        given = x if x is not None else grad_x
        K = 1 if given is None else _matrix(given, "x" if x is not None else "grad_x")[1]  # (grad_b has no K)
    code = _code(dt)
    G, gp, op = _groups(group_ptr, order, M)
    Wp = _dense_matrix(W, "W", dt, K, N, G, optional=True)
    xp, ldx = _rows(x, "x", dt, M, K, True)
    zp, ldz = _rows(z, "z", dt, M, N, True)
    yp, ldy = _rows(grad_y, "grad_y", dt, M, N)
    gxp, ldgx = _rows(grad_x, "grad_x", dt, M, K, True)
    wp, wb = _workspace(ws)
    f32 = torch.float32
    args = (M, G, gp, op, K, N, code, xp, ldx, Wp, zp, ldz, activation, yp, ldy, gxp, ldgx,
            _dense_matrix(grad_W, "grad_W", f32, K, N, G, optional=True),
            _dense(grad_b, "grad_b", f32, G * N, True), flags, wp, wb)
    _call("etp_grouped_linear_vjp", _share_device(grad_y, x, W, group_ptr, order, z, grad_x, grad_W, grad_b, ws), stream,
          args)


class TensorList:
    """Device tensors (float32 or bfloat16, contiguous, of one device) named once for many calls: the list of
    etp_grad_norm and etp_clip_grads, or the latter's outputs. It holds the tensors, whose memory must stay where it is
    (no ``set_`` or ``.data`` in between)."""

    def __init__(self, tensors):
        ts = self.tensors = tuple(tensors)
        T = torch.Tensor  # (its functions mapped: a list of 240 is checked in 0.15 ms, by comprehensions in 0.2)
        codes = list(map(_CODE.get, map(operator.attrgetter("dtype"), ts)))
        devices = set(map(T.get_device, ts))
        if None in codes or -1 in devices or not all(map(T.is_contiguous, ts)):
            for i, t in enumerate(ts):  # says which
                _code(t.dtype)
                _dense(t, f"tensor {i}", t.dtype, t.numel())
        if len(devices) > 1:
            raise ValueError(f"tensors of one call must share a device, got {sorted(devices)}")
        # etp_tensor as three words (the type in the low half of the last); their data on its own as `out`
        n = self.n = len(ts)
        self.table = numpy.empty((n, 3), dtype=numpy.int64)
        self._data = numpy.array(list(map(T.data_ptr, ts)), dtype=numpy.int64)
        self.table[:, 0], self.table[:, 1], self.table[:, 2] = self._data, list(map(T.numel, ts)), codes
        self.items, self.pointers = self.table.ctypes.data, self._data.ctypes.data
        self._shape = self.table[:, 1:].tobytes()
        self._memory = self._apart = self._clear_of = None

    def _spans(self):
        """Addresses and bytes of the tensors that are not empty."""
        if self._memory is None:
            size = self.table[:, 1] << 2 - (self.table[:, 2] != ETP_F32)
            live = size.nonzero()[0]
            self._memory = self.table[live, 0], size[live]
        return self._memory

    @property
    def apart(self):
        """Whether no two of the tensors share memory."""
        if self._apart is None:
            first, size = self._spans()
            order = first.argsort()
            self._sorted = first[order], (first + size)[order]
            self._apart = bool((self._sorted[0][1:] >= self._sorted[1][:-1]).all())
        return self._apart

    def clear_of(self, grads):
        """Whether the tensors are apart, and each is the one of its place in grads (a list of the same types and sizes) or
        shares memory with none of that list."""
        if not self.apart:
            return False
        if self._clear_of is None or self._clear_of() is not grads:
            mine, size = self._spans()
            theirs = grads._spans()[0]
            met = self._sorted[0].searchsorted(theirs + size) - self._sorted[1].searchsorted(theirs, "right")
            if (met > (mine == theirs)).any():
                return False
            self._clear_of = weakref.ref(grads)
        return True

    def like(self, other):
        """Whether the types and sizes are another list's."""
        return self._shape == other._shape


def _tensor_list(tensors):
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def etp_grad_norm_workspace(grads) -> int:
    """Bytes for etp_grad_norm and etp_clip_grads over grads (a TensorList or tensors)."""
    g = _tensor_list(grads)
    return _bytes("etp_grad_norm_workspace", g.n, g.items)


def etp_grad_norm(grads, norm, ws=None, stream=None):
    """norm (float, one element) = the 2-norm of all tensors of grads (a TensorList or tensors) taken as one vector; ws:
    etp_grad_norm_workspace(grads) bytes."""
    g = _tensor_list(grads)
    wp, wb = _workspace(ws)
    np_ = _dense(norm, "norm", torch.float32, 1)
    _call("etp_grad_norm", _share_device(norm, ws, *g.tensors[:1]), stream, (g.n, g.items, np_, wp, wb))


def etp_clip_grads(grads, max_norm: float, out=None, norm=None, ws=None, stream=None):
    """out[i] = grads[i] * min(1, max_norm / norm) with the norm of etp_grad_norm, which is written to norm (float, one
    element) when given. out: a TensorList or tensors of the same types and sizes, or None: in place. Each output is its own
    gradient or shares memory with no gradient and no other output. ws: etp_grad_norm_workspace(grads) bytes."""
    g = _tensor_list(grads)
    o = g if out is None else _tensor_list(out)
    if not o.like(g):
        raise ValueError("out must hold tensors of the types and sizes of grads")
    if not o.apart:
        raise ValueError("the clipped tensors overlap")
    if o is not g and not o.clear_of(g):
        raise ValueError("the clipped tensors overlap gradients other than their own")
    wp, wb = _workspace(ws)
    np_ = _dense(norm, "norm", torch.float32, 1, True)
    first = [t for t in (*g.tensors[:1], *o.tensors[:1], norm, ws) if t is not None]
    if not first:
        return
    _call("etp_clip_grads", _share_device(*first), stream, (g.n, g.items, max_norm, o.pointers, np_, wp, wb))

"""Host-side checks of the grouped layer, of the grouping of rows and of the
gradient norm that need no GPU: the C calls' refusals (all before any launch),
workspace sizes, the binding's tensor checks, and that every launch is checked."""
import ctypes
import os
import re

import numpy
import pytest
import torch

from equivariant_interatomic_potentials_amd import dense, etp

CSRC = os.path.join(os.path.dirname(os.path.abspath(etp.__file__)), "csrc")
INV, UNS, WS, OK = (etp.ETP_ERR_INVALID_ARGUMENT, etp.ETP_ERR_UNSUPPORTED, etp.ETP_ERR_WORKSPACE, etp.ETP_OK)
P = 256  # a non-null address that validation never reads


def rows(M=100000, G=4, ids=P, ptr=P, order=P, ws=P, wsb=1 << 40):
    return dense.lib.etp_group_rows(M, G, ids, ptr, order, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(G=0), INV), (dict(G=-3), INV), (dict(ids=None), INV), (dict(ptr=None), INV),
    (dict(order=None), INV), (dict(ids=P + 2), INV), (dict(ptr=P + 1), INV), (dict(order=P + 2), INV),
    (dict(M=0, ptr=None), INV), (dict(M=1 << 31), UNS), (dict(G=65536), UNS), (dict(ws=None), WS), (dict(ws=P + 8), WS),
    (dict(wsb=64), WS), (dict(M=10000, G=300, ws=None), WS)])
def test_group_rows_refusals(kw, want):
    assert rows(**kw) == want


def linear(M=4, G=3, ptr=P, order=None, K=8, N=16, dt=0, x=P, ldx=8, W=P, b=None, act=1, r=None, ldr=16, y=P, ldy=16,
           z=None, ldz=16):
    return dense.lib.etp_grouped_linear(M, G, ptr, order, K, N, dt, x, ldx, W, b, act, r, ldr, y, ldy, z, ldz, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(G=0), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(dt=2), INV), (dict(act=3), INV),
    (dict(act=-1), INV), (dict(ptr=None), INV), (dict(ptr=P + 2), INV), (dict(order=P + 2), INV), (dict(x=None), INV),
    (dict(W=None), INV), (dict(y=None), INV), (dict(ldx=7), INV), (dict(ldy=15), INV), (dict(r=P, ldr=15), INV),
    (dict(z=P, ldz=15), INV), (dict(x=P + 2), INV), (dict(b=P + 1), INV), (dict(y=P + 1, dt=1), INV),
    (dict(M=1 << 31), UNS), (dict(G=65536), UNS), (dict(K=65537, ldx=65537), UNS), (dict(N=65537), UNS),
    (dict(ldx=1 << 31), UNS), (dict(M=0, x=None, W=None, y=None, ptr=None), OK)])
def test_grouped_linear_refusals(kw, want):
    assert linear(**kw) == want


def vjp(M=4, G=3, ptr=P, order=None, K=8, N=16, dt=0, x=P, ldx=8, W=P, z=P, ldz=16, act=1, gy=P, ldgy=16, gx=P, ldgx=8,
        gW=P, gb=P, flags=0, ws=P, wsb=1 << 40):
    return dense.lib.etp_grouped_linear_vjp(M, G, ptr, order, K, N, dt, x, ldx, W, z, ldz, act, gy, ldgy, gx, ldgx, gW,
                                            gb, flags, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(G=0), INV), (dict(K=0), INV), (dict(dt=5), INV), (dict(act=9), INV), (dict(x=None), INV),
    (dict(W=None), INV), (dict(z=None), INV), (dict(gy=None), INV), (dict(ldgy=3), INV), (dict(ldgx=7), INV),
    (dict(ldz=15), INV), (dict(flags=2), INV), (dict(flags=4), INV), (dict(gW=P + 2), INV), (dict(gb=P + 3), INV),
    (dict(ptr=None), INV), (dict(ptr=P + 1), INV), (dict(order=P + 1), INV), (dict(M=0, ptr=None), INV),
    (dict(ws=None), WS), (dict(ws=P + 8), WS), (dict(wsb=0), WS), (dict(M=1 << 31), UNS), (dict(ldgy=1 << 31), UNS),
    (dict(G=65536), UNS), (dict(gx=None, gW=None, gb=None, gy=None), OK),
    (dict(M=0, gx=P, gW=None, gb=None, x=None, W=None, gy=None, ptr=None), OK)])
def test_grouped_linear_vjp_refusals(kw, want):
    assert vjp(**kw) == want


def tensors(*items):
    return (dense.etp_tensor * max(1, len(items)))(*(dense.etp_tensor(*i) for i in items))


GOOD = [(P, 100000, 0), (P + 2, 7, 1), (None, 0, 0)]


def norm(items=GOOD, n=None, out=P, ws=P, wsb=1 << 20, null=False):
    return dense.lib.etp_grad_norm(len(items) if n is None else n, None if null else tensors(*items), out, ws, wsb, None)


def clip(items=GOOD, n=None, most=1.0, into=None, out=P, ws=P, wsb=1 << 20, null=False):
    o = None if into is None else (ctypes.c_void_p * len(into))(*into)
    return dense.lib.etp_clip_grads(len(items) if n is None else n, None if null else tensors(*items), most, o, out, ws,
                                    wsb, None)


@pytest.mark.parametrize("call", [norm, clip])
@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INV), (dict(null=True), INV), (dict(items=[(None, 3, 0)]), INV), (dict(items=[(P, -1, 0)]), INV),
    (dict(items=[(P, 3, 2)]), INV), (dict(items=[(P + 2, 3, 0)]), INV), (dict(items=[(P + 1, 3, 1)]), INV),
    (dict(out=P + 2), INV), (dict(items=[(P, 1 << 43, 0)]), UNS), (dict(items=[(P, 1 << 43, 0), (P, 3, 7)]), INV),
    (dict(ws=None), WS), (dict(ws=P + 8), WS), (dict(wsb=0), WS)])
def test_gradient_list_refusals(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(most=-1.0), INV), (dict(most=float("nan")), INV), (dict(most=float("inf")), INV),
    (dict(into=[P, None, None]), INV), (dict(into=[P, P + 1, None]), INV), (dict(into=[P + 2, P, None]), INV),
    (dict(items=[(P, 3, 0)] * 2, into=[P, None]), INV)])
def test_clip_refusals(kw, want):
    assert clip(**kw) == want


def test_norm_needs_its_output():
    assert norm(out=None) == INV


def test_workspace_sizes():
    assert dense.etp_group_rows_workspace(0, 4) == 0
    assert dense.etp_group_rows_workspace(100, 4) == 0
    assert dense.etp_group_rows_workspace(8192, 300) == 0
    assert dense.etp_group_rows_workspace(10000, 300) >= 40000
    assert dense.etp_group_rows_workspace(1 << 20, 4) > 0
    assert dense.etp_group_rows_workspace((1 << 31) - 1, 65535) >= 4 * ((1 << 31) - 1)
    assert dense.etp_grouped_linear_vjp_workspace(0, 4, 8, 8) == 0
    assert dense.etp_grouped_linear_vjp_workspace(1000, 4, 64, 64) >= 4 * 65 * 64
    for f, args in ((dense.etp_group_rows_workspace, (-1, 4)), (dense.etp_group_rows_workspace, (4, 0)),
                    (dense.etp_group_rows_workspace, (4, 1 << 16)), (dense.etp_group_rows_workspace, (1 << 31, 4)),
                    (dense.etp_grouped_linear_vjp_workspace, (-1, 4, 8, 8)),
                    (dense.etp_grouped_linear_vjp_workspace, (8, 0, 8, 8)),
                    (dense.etp_grouped_linear_vjp_workspace, (8, 1, 0, 8)),
                    (dense.etp_grouped_linear_vjp_workspace, (8, 1, 8, 65537))):
        with pytest.raises(etp.EtpError):
            f(*args)
    assert dense.lib.etp_group_rows_workspace(1, 1, None) == INV
    assert dense.lib.etp_grouped_linear_vjp_workspace(1, 1, 1, 1, 0, None) == INV
    b = ctypes.c_size_t()
    assert dense.lib.etp_grad_norm_workspace(0, None, ctypes.byref(b)) == OK and b.value == 0
    assert dense.lib.etp_grad_norm_workspace(2, tensors((None, 1000, 0), (None, 3, 1)), ctypes.byref(b)) == OK
    assert b.value == 0
    assert dense.lib.etp_grad_norm_workspace(2, tensors((None, 1 << 20, 0), (None, 3, 1)), ctypes.byref(b)) == OK
    assert b.value > 0 and b.value % 8 == 0
    assert dense.lib.etp_grad_norm_workspace(1, tensors((None, 5, 0)), None) == INV
    assert dense.lib.etp_grad_norm_workspace(1, tensors((None, -5, 0)), ctypes.byref(b)) == INV


def test_binding_refuses_host_and_mismatched_tensors():
    x, W, y, ptr = torch.zeros(4, 8), torch.zeros(3, 8, 16), torch.zeros(4, 16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        dense.etp_grouped_linear(x, W, y, ptr)
    with pytest.raises(ValueError, match="group_ptr must be"):
        dense.etp_grouped_linear(x, W, y, ptr.long())
    with pytest.raises(ValueError, match="features must be"):
        dense.etp_grouped_linear(x.double(), W, y, ptr)
    with pytest.raises(ValueError, match="2-D"):
        dense.etp_grouped_linear(x[0], W, y, ptr)
    with pytest.raises(ValueError, match="groups"):
        dense.etp_grouped_linear_vjp(x, W[0], y, ptr)
    with pytest.raises(ValueError, match="ids must be"):
        dense.etp_group_rows(ptr.long(), ptr, ptr)
    with pytest.raises(ValueError, match="device tensor"):
        dense.TensorList([x])
    with pytest.raises(ValueError, match="contiguous"):
        dense.TensorList([W[:, :, 0]])
    with pytest.raises(ValueError, match="features must be"):
        dense.TensorList([ptr])


def listed(*rows):
    """A list that claims tensors (address, entries, type) without owning any."""
    t = dense.TensorList([])
    t.n, t.table = len(rows), numpy.array(rows, dtype=numpy.int64).reshape(-1, 3)
    t._shape = t.table[:, 1:].tobytes()
    return t


def test_gradient_lists():
    """The list is etp_tensor's layout, and knows whether its tensors share memory."""
    assert ctypes.sizeof(dense.etp_tensor) == 24 and dense.etp_tensor.dtype.offset == 16
    t = listed((256, 10, 0), (4096, 7, 1))
    item = ctypes.cast(t.table.ctypes.data, ctypes.POINTER(dense.etp_tensor))[1]
    assert (item.data, item.numel, item.dtype) == (4096, 7, 1)
    assert t.like(listed((0, 10, 0), (8, 7, 1))) and not t.like(listed((256, 10, 0)))
    assert not t.like(listed((256, 10, 0), (4096, 7, 0))) and not t.like(listed((256, 11, 0), (4096, 7, 1)))
    assert listed().apart and listed((256, 10, 0)).apart
    assert listed((296, 10, 1), (256, 10, 0), (316, 1, 0)).apart  # 40, 20 and 4 bytes side by side
    assert not listed((295, 10, 1), (256, 10, 0)).apart and not listed((256, 10, 0), (256, 10, 0)).apart
    assert listed((256, 10, 0), (256, 0, 0), (260, 0, 1)).apart
    with pytest.raises(ValueError, match="types and sizes"):
        dense.etp_clip_grads([], 1.0, listed((256, 3, 0)))
    with pytest.raises(ValueError, match="overlap"):
        dense.etp_clip_grads(listed((256, 3, 0), (260, 3, 0)), 1.0)


def test_every_launch_is_checked():
    """A refused launch is reported by the call that made it: hipGetLastError follows each launch before the next one."""
    files = ("etp_grouped.hip", "etp_grouped_vjp.hip", "etp_group_rows.hip", "etp_grad_norm.hip")
    for f in files:
        text = open(os.path.join(CSRC, f)).read()
        launches = [m.end() for m in re.finditer(r"hipLaunchKernelGGL\(", text)]
        assert launches
        for at in launches:
            rest = text[at:]
            check, other = rest.find("hipGetLastError"), re.search(r"hipFuncSetAttribute|hipLaunchKernelGGL|\n}\n", rest)
            stop = other.start() if other else len(rest)
            assert 0 <= check < stop, (f, text[:at].count("\n") + 1)

"""Host-side checks of the dense operators that need no GPU: the exported ABI,
the C calls' refusals (all before any launch), workspace sizes, and the
binding's tensor checks."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from equivariant_interatomic_potentials_amd import dense, etp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, WS, OK = (etp.ETP_ERR_INVALID_ARGUMENT, etp.ETP_ERR_UNSUPPORTED, etp.ETP_ERR_WORKSPACE, etp.ETP_OK)
P = 256  # a non-null address that validation never reads


def test_header_symbols_exported():
    text = open(os.path.join(ROOT, "include", "etp_dense.h")).read()
    names = sorted(set(re.findall(r"ETP_API\s+[\w\s\*]+?\b(etp_\w+)\s*\(", text)))
    assert names == sorted(dense.ABI_SYMBOLS)
    out = subprocess.run(["nm", "-D", "--defined-only", etp._LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r" T (etp_\w+)$", out, flags=re.M))


def linear(M=4, K=8, N=16, dt=0, x=P, ldx=8, W=P, b=None, act=1, r=None, ldr=16, y=P, ldy=16, z=None, ldz=16):
    return dense.lib.etp_linear(M, K, N, dt, x, ldx, W, b, act, r, ldr, y, ldy, z, ldz, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(dt=2), INV), (dict(act=3), INV), (dict(act=-1), INV),
    (dict(x=None), INV), (dict(W=None), INV), (dict(y=None), INV), (dict(ldx=7), INV), (dict(ldy=15), INV),
    (dict(r=P, ldr=15), INV), (dict(z=P, ldz=15), INV), (dict(x=P + 2), INV), (dict(b=P + 1), INV),
    (dict(y=P + 1, dt=1), INV), (dict(M=1 << 31), UNS), (dict(K=65537, ldx=65537), UNS), (dict(N=65537), UNS),
    (dict(ldx=1 << 31), UNS), (dict(M=0, x=None, W=None, y=None), OK)])
def test_linear_refusals(kw, want):
    assert linear(**kw) == want


def linear_vjp(M=4, K=8, N=16, dt=0, x=P, ldx=8, W=P, z=P, ldz=16, act=1, gy=P, ldgy=16, gx=P, ldgx=8, gW=P, gb=P,
               flags=0, ws=P, wsb=1 << 40):
    return dense.lib.etp_linear_vjp(M, K, N, dt, x, ldx, W, z, ldz, act, gy, ldgy, gx, ldgx, gW, gb, flags, ws, wsb,
                                    None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(K=0), INV), (dict(dt=5), INV), (dict(act=9), INV), (dict(x=None), INV),
    (dict(W=None), INV), (dict(z=None), INV), (dict(gy=None), INV), (dict(ldgy=3), INV), (dict(ldgx=7), INV),
    (dict(ldz=15), INV), (dict(flags=2), INV), (dict(flags=4), INV), (dict(gW=P + 2), INV), (dict(gb=P + 3), INV),
    (dict(ws=None), WS), (dict(ws=P + 8), WS), (dict(wsb=0), WS), (dict(M=1 << 31), UNS),
    (dict(ldgy=1 << 31), UNS)])
def test_linear_vjp_refusals(kw, want):
    assert linear_vjp(**kw) == want


def norm(M=4, C=8, dt=0, x=P, ldx=8, g=None, b=None, eps=1e-5, y=P, ldy=8, mean=None, rstd=None):
    return dense.lib.etp_layer_norm(M, C, dt, x, ldx, g, b, eps, y, ldy, mean, rstd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(C=0), INV), (dict(dt=-1), INV), (dict(x=None), INV), (dict(y=None), INV),
    (dict(ldx=7), INV), (dict(ldy=7), INV), (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(g=P + 2), INV), (dict(mean=P + 1), INV), (dict(C=65537, ldx=65537), UNS),
    (dict(M=1 << 31), UNS), (dict(M=0, x=None, y=None), OK)])
def test_layer_norm_refusals(kw, want):
    assert norm(**kw) == want


def norm_vjp(M=4, C=8, dt=0, x=P, ldx=8, g=P, mean=P, rstd=P, gy=P, ldgy=8, gx=P, ldgx=8, gg=P, gb=P, flags=0, ws=P,
             wsb=1 << 40):
    return dense.lib.etp_layer_norm_vjp(M, C, dt, x, ldx, g, mean, rstd, gy, ldgy, gx, ldgx, gg, gb, flags, ws, wsb,
                                        None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(C=0), INV), (dict(mean=None), INV), (dict(rstd=None), INV), (dict(x=None), INV),
    (dict(gy=None), INV), (dict(ldgx=7), INV), (dict(flags=2), INV), (dict(gg=P + 2), INV), (dict(ws=None), WS),
    (dict(ws=P + 4), WS), (dict(wsb=8), WS), (dict(M=1 << 31), UNS)])
def test_layer_norm_vjp_refusals(kw, want):
    assert norm_vjp(**kw) == want


def orth(n=2, r=8, c=16, dt=0, G=P, steps=5, coef=None, eps=1e-7, X=P, ws=P, wsb=1 << 40):
    f = None if coef is None else (ctypes.c_float * 3)(*coef)
    return dense.lib.etp_orthogonalize(n, r, c, dt, G, steps, f, eps, X, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INV), (dict(r=0), INV), (dict(c=0), INV), (dict(dt=3), INV), (dict(G=None), INV), (dict(X=None), INV),
    (dict(steps=0), INV), (dict(steps=65), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV),
    (dict(coef=(1.0, float("inf"), 0.0)), INV), (dict(ws=None), WS), (dict(ws=P + 8), WS), (dict(wsb=16), WS),
    (dict(n=65536), UNS), (dict(r=65537), UNS), (dict(n=0, G=None, X=None, ws=None), OK)])
def test_orthogonalize_refusals(kw, want):
    assert orth(**kw) == want


def test_workspace_sizes():
    assert dense.etp_linear_vjp_workspace(0, 8, 8) == 0
    assert dense.etp_linear_vjp_workspace(1000, 64, 64) >= 4 * 65 * 64
    assert dense.etp_layer_norm_vjp_workspace(0, 8) == 0
    assert dense.etp_layer_norm_vjp_workspace(1000, 64) >= 8 * 64
    assert dense.etp_orthogonalize_workspace(0, 8, 8) == 0
    assert dense.etp_orthogonalize_workspace(3, 8, 9) > 0
    for args in ((-1, 8, 8), (8, 0, 8), (8, 8, 0)):
        with pytest.raises(etp.EtpError):
            dense.etp_linear_vjp_workspace(*args)
    with pytest.raises(etp.EtpError):
        dense.etp_layer_norm_vjp_workspace(5, 0)
    with pytest.raises(etp.EtpError):
        dense.etp_orthogonalize_workspace(1, 0, 4)
    for f in ("etp_linear_vjp_workspace", "etp_orthogonalize_workspace"):
        assert getattr(dense.lib, f)(1, 1, 1, 0, None) == INV
    assert dense.lib.etp_layer_norm_vjp_workspace(1, 1, 0, None) == INV


def test_binding_refuses_host_and_mismatched_tensors():
    x, W, y = torch.zeros(4, 8), torch.zeros(8, 16), torch.zeros(4, 16)
    with pytest.raises(ValueError, match="device tensor"):
        dense.etp_linear(x, W, y)
    with pytest.raises(ValueError, match="features must be"):
        dense.etp_linear(x.double(), W, y)
    with pytest.raises(ValueError, match="2-D"):
        dense.etp_linear(x[0], W, y)
    with pytest.raises(ValueError, match="x is required"):
        dense._rows(None, "x", torch.float32, 1, 1)
    with pytest.raises(ValueError, match="must be"):
        dense._rows(x, "x", torch.bfloat16, 4, 8)
    with pytest.raises(ValueError, match=r"\[4\]\[9\]"):
        dense._rows(x, "x", torch.float32, 4, 9)
    with pytest.raises(ValueError, match="\\[rows\\]\\[cols\\]"):
        dense.etp_orthogonalize(x[0], x[0])

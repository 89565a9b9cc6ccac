"""Float64 definitions of the dense operators (torch on the CPU), the
reference of tests/test_gpu_dense_*.py and tests/test_dense_host.py."""
from __future__ import annotations

import math

import torch

ACTS = {"none": 0, "silu": 1, "gelu": 2}


def act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return z


def act_slope(name, z):
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def f64(t):
    return None if t is None else t.detach().cpu().double()


def linear(x, W, bias=None, name="none", res=None):
    z = f64(x) @ f64(W)
    if bias is not None:
        z = z + f64(bias)
    y = act(name, z)
    return (y if res is None else y + f64(res)), z


def linear_vjp(x, W, gy, z, name):
    d = f64(gy)
    if name != "none":
        d = d * act_slope(name, f64(z))
    return d @ f64(W).T, f64(x).T @ d, d.sum(0)


def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    x = f64(x)
    mean = x.mean(1)
    rstd = ((x - mean[:, None]) ** 2).mean(1).add(eps).rsqrt()
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * f64(gamma)
    if beta is not None:
        y = y + f64(beta)
    return y, mean, rstd


def layer_norm_vjp(x, mean, rstd, gy, gamma=None):
    r = f64(rstd)[:, None]
    h = (f64(x) - f64(mean)[:, None]) * r
    g = f64(gy)
    d = g if gamma is None else g * f64(gamma)
    gx = r * (d - d.mean(1, keepdim=True) - h * (d * h).mean(1, keepdim=True))
    return gx, (g * h).sum(0), g.sum(0)


def orthogonalize(G, steps=5, coef=(3.4445, -4.7750, 2.0315), eps=1e-7):
    X = f64(G)
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.mT
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in coef)
    for _ in range(steps):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.mT if tall else X


def close(got, ref, scale=None, tol=1e-5):
    """Elementwise bound for an output of the got tensor's type: tol of the largest |ref| (or of `scale`) for float
    arithmetic, plus half a unit in the last place of bf16 (2^-8 |ref|) where the output is stored in bf16. A shape,
    NaN or infinity mismatch fails."""
    assert got.shape == ref.shape, (got.shape, ref.shape)
    g = f64(got)
    if ref.numel() == 0:
        return
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(g))
    bound = tol * float(ref[fin].abs().max() if scale is None else scale) if fin.any() else 0.0
    lim = torch.full_like(ref, bound)
    if got.dtype == torch.bfloat16:
        lim = lim + ref.abs() * 2.0 ** -8
    bad = (g - ref).abs()[fin] > lim[fin]
    assert not bad.any(), (int(bad.sum()), float(((g - ref).abs()[fin] / (lim[fin] + 1e-300)).max()))

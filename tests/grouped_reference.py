"""Float64 definitions of the grouped layer, of the grouping of rows and of the
gradient norm (torch and numpy on the CPU), the reference of
tests/test_gpu_grouped_*.py and tests/test_gpu_grad_norm.py."""
from __future__ import annotations

import numpy as np
import torch

import dense_reference as ref


def group_rows(ids, n_groups):
    """(group_ptr, order) as numpy int32."""
    ids = np.asarray(ids)
    key = np.where((ids < 0) | (ids >= n_groups), n_groups, ids).astype(np.int64)
    ptr = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=n_groups + 1)[:n_groups])])
    return ptr.astype(np.int32), np.argsort(key, kind="stable").astype(np.int32)


def rows_of(ptr, order, rows):
    """The row numbers of each group (long tensors on the CPU)."""
    o = torch.arange(rows) if order is None else order.detach().cpu().long()
    p = [int(v) for v in ptr]
    return [o[p[g]:p[g + 1]] for g in range(len(p) - 1)]


def linear(x, W, ptr, order=None, bias=None, name="none", res=None, y0=None, z0=None):
    """(y, z): y0 and z0 where a row is in no group."""
    M, N = x.shape[0], W.shape[-1]
    new = lambda t: torch.full((M, N), float("nan"), dtype=torch.float64) if t is None else ref.f64(t).clone()
    y, z = new(y0), new(z0)
    x, res = ref.f64(x), ref.f64(res)
    for g, r in enumerate(rows_of(ptr, order, M)):
        y[r], z[r] = ref.linear(x[r], W[g], None if bias is None else bias[g], name, None if res is None else res[r])
    return y, z


def linear_vjp(x, W, gy, ptr, order=None, z=None, name="none", gx0=None):
    M, (G, K, N) = gy.shape[0], W.shape
    gx = torch.full((M, K), float("nan"), dtype=torch.float64) if gx0 is None else ref.f64(gx0).clone()
    gW, gb = torch.zeros(G, K, N, dtype=torch.float64), torch.zeros(G, N, dtype=torch.float64)
    x, gy, z = ref.f64(x), ref.f64(gy), ref.f64(z)
    for g, r in enumerate(rows_of(ptr, order, M)):
        gx[r], gW[g], gb[g] = ref.linear_vjp(x[r], W[g], gy[r], None if z is None else z[r], name)
    return gx, gW, gb


def linear_vjp_terms(x, W, gy, ptr, order=None, z=None, name="none"):
    """Largest 2-norm of the terms of one entry of gx, gW and gb.

    The bar of a float sum whose terms have either sign. The kernels add at most 256 results of the matrix instruction
    on top of each other, which drops up to a unit (2^-23) of the partial sum each time, half of one on average and to
    the same side. A partial sum of i terms of n is about sqrt(i / n) |t|, so that 256 results lose about
    2 / 3 * 256 * 2^-24 |t| = 1e-5 |t| of their chain, and a gradient of several chains, or one of fewer results, less.
    (Terms of one sign have a larger bound of their own: test_gpu_grouped_sums.) Where terms cancel the sum itself is
    far smaller than |t| and no bar."""
    M, (G, K, N) = gy.shape[0], W.shape
    x, gy, z = ref.f64(x), ref.f64(gy), ref.f64(z)
    most = [0.0, 0.0, 0.0]
    for g, r in enumerate(rows_of(ptr, order, M)):
        if len(r):
            d2 = (gy[r] if name == "none" else gy[r] * ref.act_slope(name, z[r])).square()
            sums = (d2 @ ref.f64(W[g]).square().T, x[r].square().T @ d2, d2.sum(0))
            most = [max(m, float(s.max()) ** 0.5) for m, s in zip(most, sums)]
    return most


def grad_norm(tensors):
    return float(sum(float(ref.f64(t).square().sum()) for t in tensors) ** 0.5)

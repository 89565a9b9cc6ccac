"""GPU parity of the linear layer at row counts that fill the chip with tiles
of each kind: contractions above 128 in tiles of 128 and of 32 columns, 64 and
128 rows, and gradients cut into splits that do not divide the panels. Bounds
as in test_gpu_dense_linear.py: 1e-5 of the largest entry (products of 2^-22
and float sums of at most 2^10 terms a partial set, the sets added pairwise:
well below it), plus half a bf16 unit where the output is bf16."""
import pytest

import dense_reference as ref
from test_gpu_dense_linear import TYPES, make, out, run_vjp, say

pytestmark = pytest.mark.gpu

SHAPES = [(16500, 200, 7), (16399, 129, 32), (66001, 130, 5), (16500, 140, 150), (40003, 260, 33), (33000, 300, 200)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward_tiles(M, K, N, dtype):
    from equivariant_interatomic_potentials_amd import dense
    say("linear", M, K, N, dtype)
    p = make(M, K, N, dtype, M + K + N, 1)
    y, z = out(M, N, p["dt"], 1, 7.0), out(M, N, p["dt"], 1, 7.0)
    dense.etp_linear(p["x"], p["W"], y, p["b"], ref.ACTS["silu"], p["res"], z)
    yr, zr = ref.linear(p["x"], p["W"], p["b"], "silu", p["res"])
    ref.close(y, yr)
    ref.close(z, zr)
    assert (y._base[:, N:] == 7.0).all() and (z._base[:, N:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("M,N,K", SHAPES)  # the input gradient contracts along N
def test_vjp_tiles(M, N, K, act, dtype):
    say("linear_vjp", M, K, N, dtype, act)
    p = make(M, K, N, dtype, 3 * M + K + N)
    for g, r in zip(run_vjp(p, act, M, K, N), ref.linear_vjp(p["x"], p["W"], p["gy"], p["z"], act)):
        ref.close(g, r)


def test_accumulate_tiles():
    import torch
    M, K, N = 16500, 7, 200
    say("linear_vjp accumulate", M, K, N)
    p = make(M, K, N, "f32", 5)
    base = [torch.randn(M, K, device="cuda"), torch.randn(K, N, device="cuda"), torch.randn(N, device="cuda")]
    want = [b.double().cpu() + r.double().cpu()
            for b, r in zip(base, ref.linear_vjp(p["x"], p["W"], p["gy"], p["z"], "silu"))]
    from equivariant_interatomic_potentials_amd import etp
    for g, r in zip(run_vjp(p, "silu", M, K, N, flags=etp.ETP_FLAG_ACCUMULATE, base=base), want):
        ref.close(g, r)

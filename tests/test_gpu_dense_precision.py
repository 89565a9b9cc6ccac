"""The dense operators' arithmetic, held to what a float can do rather than to a
fraction of the largest entry."""
import pytest

import dense_reference as ref
from test_gpu_dense_linear import out, workspace

pytestmark = pytest.mark.gpu

TYPES = ["f32", "bf16"]


def say(*a):
    print("[case]", *a, flush=True)


@pytest.mark.parametrize("M,N,K", [(2000, 64, 64), (2000, 128, 40), (600, 300, 40), (17000, 300, 40), (600, 300, 200),
                                   (17000, 300, 200)])
def test_input_gradient_of_a_bf16_layer(M, N, K):
    """grad_x of nearly equal d of opposite weights: the difference is held to 2^-19 of d (the slope's own error: a few
    units of the logistic function times 1 + z) and the result's rounding, so that d has to keep its float's bits."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("bf16 grad_x", M, K, N)
    g = torch.Generator().manual_seed(M + N + K)
    z = (0.25 + 0.75 * torch.rand(2 * M, generator=g)).bfloat16()
    gy = (1 + torch.rand(2 * M, generator=g)).bfloat16()
    order = torch.argsort(gy.double() * ref.act_slope("silu", z.double()))
    z, gy = z[order].view(M, 2), gy[order].view(M, 2)  # rows of two neighbours
    mix = torch.randperm(M, generator=g)
    r, j = torch.arange(M), 2 * (torch.arange(M) % (N // 2))
    zz, gg = torch.zeros(M, N, dtype=torch.bfloat16), torch.zeros(M, N, dtype=torch.bfloat16)
    for i in range(2):
        zz[r, j + i], gg[r, j + i] = z[mix, i], gy[mix, i]
    W = torch.tensor([1.0, -1.0]).repeat(N // 2).bfloat16()[None].expand(K, N).contiguous()
    gx, alone = out(M, K, torch.bfloat16), out(M, K, torch.bfloat16)
    gW = torch.empty(K, N, device="cuda")
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    dense.etp_linear_vjp(x, W.cuda(), gg.cuda(), zz.cuda(), 1, gx, gW, None, workspace(M, K, N, torch.bfloat16))
    dense.etp_linear_vjp(None, W.cuda(), gg.cuda(), zz.cuda(), 1, alone)
    d = gg.double() * ref.act_slope("silu", zz.double())
    want = (d @ W.double().T)
    lim = 2.0 ** -19 * d.abs().sum(1, keepdim=True) + 2.0 ** -8 * want.abs()
    for t in (gx, alone):
        err = (ref.f64(t) - want).abs()
        assert (err <= lim).all(), (int((err > lim).sum()), float((err / lim).max()))


@pytest.mark.parametrize("r,c", [(128, 128), (60, 500), (200, 300), (300, 200)])
def test_orthogonalised_bf16_is_rounded_once(r, c):
    """bf16 matrices of one strong direction, whose steps amplify what is lost on the way by up to a^5 = 485. With float
    quality in between (a unit of 2^-24 of |X| amplified: sigma) an entry ends on another bf16 value than the float64
    result's only where that lies within a few sigma of a tie: at most 2 sigma / ulp of the entries of one size."""
    import torch
    from test_gpu_dense_orth import run
    say("orth bf16", r, c)
    g = torch.Generator().manual_seed(r + c)
    G = (torch.randn(r, 1, generator=g) @ torch.randn(1, c, generator=g) + 1e-3 * torch.randn(r, c, generator=g)).bfloat16()
    want = ref.orthogonalize(G)
    X = ref.f64(run(G.cuda()))
    sigma = 485 * 2.0 ** -24 * float(want.square().mean().sqrt())
    ulp = torch.exp2(torch.floor(torch.log2(want.abs().clamp_min(1e-30))) - 7)
    limit = float((2 * sigma / ulp).clamp_max(1.0).sum())
    off = int((X != want.bfloat16().double()).sum())
    assert off <= limit, (off, limit, want.numel())

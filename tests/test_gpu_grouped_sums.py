"""The weight gradients of the grouped layer where the sums are long, or one workgroup forms them alone."""
import pytest

import dense_reference as ref
import grouped_reference as gref

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16"]


def say(*a):
    print("[case]", *a, flush=True)


def dtype_of(name):
    import torch
    return torch.float32 if name == "f32" else torch.bfloat16


def call(x, W, gy, ptr, order, z, act, gx, gW, gb, flags=0):
    """The VJP with a workspace of exactly the bytes it asks for; what lies behind them stays."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    G, N = ptr.numel() - 1, gy.shape[1]
    K = x.shape[1] if x is not None else W.shape[1]
    size = dense.etp_grouped_linear_vjp_workspace(gy.shape[0], G, K, N, gy.dtype)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    dense.etp_grouped_linear_vjp(x, W, gy, ptr, order, z, ref.ACTS[act], gx, gW, gb, ws[:size] if size else None, flags)
    torch.cuda.synchronize()
    assert (ws[size:] == 0xFF).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,G,K,N", [(2, 1, 64, 64), (31, 1, 128, 128), (300, 3, 2048, 2048), (70, 1, 1500, 4096)])
def test_one_run_holds_every_group(M, G, K, N, dtype):
    """Small calls, and matrices of so many blocks that each has one workgroup: no partial sums, and no room for them."""
    import torch
    say("grouped one run", M, G, K, N, dtype)
    dt, g = dtype_of(dtype), torch.Generator().manual_seed(M + K)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()
    x, gy, z = rnd(M, K).to(dt), rnd(M, N).to(dt), rnd(M, N).to(dt)
    W = (rnd(G, K, N) / K ** 0.5).to(dt)
    ptr = torch.linspace(0, M, G + 1).int().cuda()
    order = torch.randperm(M, generator=g).int().cuda()
    for act in ("silu", "none"):
        gx, gW, gb = torch.empty_like(x), torch.empty(G, K, N, device="cuda"), torch.empty(G, N, device="cuda")
        call(x, W, gy, ptr, order, z if act != "none" else None, act, gx, gW, gb)
        want = gref.linear_vjp(x, W, gy, ptr, order, z, act)
        terms = gref.linear_vjp_terms(x, W, gy, ptr, order, z, act)
        for a, b, t in zip((gx, gW, gb), want, terms):
            ref.close(a, b, scale=max(t, float(b.abs().max())))

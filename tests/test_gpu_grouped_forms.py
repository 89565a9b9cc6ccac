"""GPU parity of every form of the grouped layer's kernels with float64: the calls of grouped_shapes, which between them
take each compiled kernel, through an order and with rows in no group."""
import pytest

import dense_reference as ref
import grouped_shapes as shapes
import test_gpu_grouped_linear as base

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,G,K,N", shapes.FORWARD)
def test_forward(M, G, K, N, dtype):
    act = ["gelu", "none", "silu"][(M + G + K + N) % 3]
    base.say("grouped form", sorted(map(str, shapes.forward(dtype == "f32", M, G, K, N))), M, G, K, N, act)
    p = base.make(M, G, K, N, dtype, M + K + N)
    o7 = base.out(M, N, p["dt"])
    for got, want in zip(base.run_fwd(p, act, M, N), base.want_fwd(p, act, o7, o7)):
        ref.close(got, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("M,G,K,N", shapes.VJP)
def test_vjp(M, G, K, N, act, dtype):
    base.say("grouped form", sorted(map(str, shapes.vjp(dtype == "f32", act, M, G, K, N))), M, G, K, N, act)
    p = base.make(M, G, K, N, dtype, M + K + N)
    base.close_vjp(base.run_vjp(p, act, M, K, N), p, act, base.out(M, K, p["dt"]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["gelu", "none"])
def test_accumulates_where_parts_are_joined_by_boundaries(act, dtype):
    """More groups than four times the runs: the parts of a group that crosses runs are found from the boundary."""
    import torch
    from equivariant_interatomic_potentials_amd import etp
    sizes = [(i * 7) % 4 for i in range(2000)]  # a quarter of them empty
    sizes[700], sizes[1500] = 5000, 1501
    M, G, K, N = sum(sizes), len(sizes), 200, 150
    base.say("grouped accumulate", M, G, K, N, dtype, act)
    p = base.make(M, G, K, N, dtype, 9, pad=0)
    p["ptr"] = torch.tensor([0, *sizes]).cumsum(0).int().cuda()
    g = torch.Generator().manual_seed(2)
    to = (torch.randn(M, K, generator=g).to(p["dt"]).cuda(), torch.randn(G, K, N, generator=g).cuda(),
          torch.randn(G, N, generator=g).cuda())
    was = [ref.f64(t) for t in to]
    got = base.run_vjp(p, act, M, K, N, flags=etp.ETP_FLAG_ACCUMULATE, base=to)
    for t, b, r in zip(got, was, base.want_vjp(p, act, torch.zeros(M, K))):
        ref.close(t, b + r)


@pytest.mark.parametrize("K,N", [(64, 64), (200, 300)])
def test_infinite_bf16_gradients_without_activation(K, N):
    """d is grad_y as it is, one part: an infinity stays one, as in IEEE arithmetic."""
    import torch
    M, G = 400, 4
    base.say("grouped infinite", K, N)
    p = base.make(M, G, K, N, "bf16", 4, pad=0)
    row = int(p["order"][int(p["ptr"][2])])  # the first row of group 2
    p["gy"][row, 1] = float("-inf")
    got = base.run_vjp(p, "none", M, K, N)
    for g, r in zip(got, base.want_vjp(p, "none", base.out(M, K, p["dt"]))):
        ref.close(g, r)
        inf = torch.isinf(r)
        assert inf.any() and torch.equal(ref.f64(g)[inf], r[inf])

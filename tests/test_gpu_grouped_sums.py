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
    K = 1 if x is None and W is None else x.shape[1] if x is not None else W.shape[1]
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


# What a sum of terms of one sign may be off by, relative to itself, in halves of a unit (2^-24). The kernel adds at most 256
# results of the matrix instruction to an accumulator (six for 32 rows of a float layer, 1344 rows; three for 32 of a bf16
# layer with an activation, 2688; one without, 8192). The i-th of n like terms is off by at most a whole unit (the instruction
# may cut off) of the partial sum, which is i / n of the result: 256 halves. At most 32 such chains are added in float, each
# with half a unit: 16. Parts of a group are joined in double. The slope of the activation is good to 8 halves, the parts'
# dropped products, the result's own rounding and one more addition take 8. (The bias gradient adds at most 512 values and 16
# sums with half a unit each, 264, and has no products.)
STEP = 2.0 ** -24
LONG = (256 + 16 + 8 + 8) * STEP


def slope64(act, z):
    return ref.act_slope(act, z.double())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("sizes,K,N", [([150000, 7, 50001], 1024, 1024), ([100003], 2048, 2048), ([3000001], 64, 64),
                                       ([200000, 0, 150001, 33], 128, 96), ([70000, 30001], 40, 1500)])
def test_long_sums_of_rows_that_are_alike(sizes, K, N, act, dtype):
    """The rows of a perfect crystal: every term of a sum is the same, so that its roundings are too."""
    import torch
    M, G = sum(sizes), len(sizes)
    say("grouped alike", sizes, K, N, act, dtype)
    dt, g = dtype_of(dtype), torch.Generator().manual_seed(K + N)
    row = lambda n: (0.5 + 2.0 * torch.rand(n, generator=g)).to(dt).cuda()
    u, v, w = row(K), row(N), row(N)
    x, gy, z = (t.expand(M, -1).contiguous() for t in (u, v, w))
    ptr = torch.tensor([0, *sizes]).cumsum(0).int().cuda()
    d = v.double() if act == "none" else v.double() * slope64(act, w)
    n = torch.tensor(sizes, device="cuda").double()
    want_b = n[:, None] * d
    want_W = n[:, None, None] * u.double()[:, None] * d
    for flags in (0, 1):
        gW = torch.rand(G, K, N, generator=g).cuda() * 1000
        gb = torch.rand(G, N, generator=g).cuda() * 1000
        was_W, was_b = (gW.double(), gb.double()) if flags else (0.0, 0.0)
        call(x, None, gy, ptr, None, z if act != "none" else None, act, None, gW, gb, flags)
        for got, want in ((gW, want_W + was_W), (gb, want_b + was_b)):
            off = ((got.double() - want).abs() / want.clamp(min=1e-30)).max()
            print("   off by", float(off), flush=True)
            assert off <= LONG
        alone = torch.full((G, N), 7.0, device="cuda")
        call(None, None, gy, ptr, None, z if act != "none" else None, act, None, None, alone)
        assert ((alone.double() - want_b).abs() <= LONG * want_b).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["gelu", "none"])
@pytest.mark.parametrize("M,G,K,N", [(100000, 2, 1024, 1024), (1000003, 5, 64, 128)])
def test_long_sums_of_one_sign(M, G, K, N, act, dtype):
    """Terms of one sign that differ, through an order, in groups that cross workgroups."""
    import torch
    say("grouped one sign", M, G, K, N, act, dtype)
    dt, g = dtype_of(dtype), torch.Generator(device="cuda").manual_seed(M + K)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").abs().to(dt)
    x, gy, z = rnd(M, K), rnd(M, N), rnd(M, N)
    edges = torch.linspace(0, 1, G + 1) ** 2 * M
    ptr = edges.int().cuda()
    order = torch.randperm(M, generator=g, device="cuda").int()
    gW, gb = torch.empty(G, K, N, device="cuda"), torch.empty(G, N, device="cuda")
    call(x, None, gy, ptr, order, z if act != "none" else None, act, None, gW, gb)
    for k in range(G):
        r = order[int(ptr[k]):int(ptr[k + 1])].long()
        d = gy[r].double() if act == "none" else gy[r].double() * slope64(act, z[r])
        for got, want in ((gW[k], x[r].double().t().contiguous() @ d), (gb[k], d.sum(0))):
            off = ((got.double() - want).abs() / want.clamp(min=1e-30)).max()
            print("   off by", float(off), flush=True)
            assert off <= LONG

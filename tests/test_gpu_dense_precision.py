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


# One non-zero term in every sum: an output is a product of two floats of which
# six partial products are added. The dropped ones are at most 2^-24 of it (a
# part is below 2^-8 and the next below 2^-17 of the value, in two pairs), the
# last addition rounds by 2^-23 at most (half of that to nearest), and the
# earlier ones by 2^-8 of that: together below 1.6 * 2^-23. Two parts, or three
# truncated ones, miss it at the mantissas tried here.
ONE_PRODUCT = 1.6 * 2.0 ** -23


def mantissas(n, seed):
    """Floats of either sign and exponents of -12 .. 12; half of them with bits in the places that a part's rounding or
    truncation costs most, the others random."""
    import torch
    g = torch.Generator().manual_seed(seed)
    u = lambda k: 2.0 ** -k
    hard = torch.tensor([1 + u(7) - u(23), 1 + u(8) - u(23), 1 + u(8) + u(23), 1 + u(7) - u(15) - u(23), 1 + u(8) - u(16) - u(23),
                         1 + u(8) + u(17) - u(23), 1 + u(9) + u(16), 1 + u(15) - u(23), 1 + u(16) + u(23), 2 - u(23)])
    pick = hard[torch.randint(len(hard), (n,), generator=g)]
    rand = 1 + torch.randint(1 << 23, (n,), generator=g).float() * u(23)
    v = torch.where(torch.rand(n, generator=g) < 0.5, pick, rand)
    sign = 1 - 2 * torch.randint(2, (n,), generator=g).float()
    return v * sign * torch.exp2(torch.randint(-12, 13, (n,), generator=g).float())


def one_per_row(M, K, seed):
    """[M, K] with one non-zero in every row, in column r % K."""
    import torch
    x = torch.zeros(M, K)
    r = torch.arange(M)
    x[r, r % K] = mantissas(M, seed)
    return x


def check_products(got, want, what):
    err = (ref.f64(got) - want).abs()
    bad = err > ONE_PRODUCT * want.abs()
    assert not bad.any(), (what, int(bad.sum()), float((err / want.abs().clamp_min(1e-300)).max()) * 2.0 ** 23)


# resident matrix of 32, 64, 96 and 128 inputs; few rows of a long contraction; tiles of 32, 64 and 128 columns by 64
# and 128 rows
FORWARD = [(300, 32, 64), (300, 50, 130), (2000, 96, 128), (260, 128, 257), (130, 300, 65), (16500, 140, 30),
           (66000, 130, 20), (16500, 140, 64), (66000, 130, 64), (16500, 140, 130), (40000, 130, 200)]


@pytest.mark.parametrize("M,K,N", FORWARD)
def test_single_products_forward(M, K, N):
    from equivariant_interatomic_potentials_amd import dense
    import torch
    say("single products", M, K, N)
    x, W = one_per_row(M, K, M), mantissas(K * N, N).view(K, N)
    y = out(M, N, torch.float32)
    dense.etp_linear(x.cuda(), W.cuda(), y)
    r = torch.arange(M) % K
    check_products(y, x.double().sum(1, keepdim=True) * W.double()[r], "y")


# every block of the panel kernel, gradients in blocks, and input gradients as products of their own
VJP = [(300, 32, 32), (300, 20, 64), (300, 32, 128), (300, 64, 30), (400, 64, 64), (300, 64, 128), (300, 128, 32),
       (300, 128, 64), (2000, 128, 128), (500, 200, 100), (500, 100, 200), (700, 260, 300), (17000, 200, 140),
       (17000, 140, 200)]


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("M,K,N", VJP)
def test_single_products_vjp(M, K, N, act):
    """With SiLU, z = 0: its slope is one half exactly, and d = gy / 2."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("single products, VJP", M, K, N, act)
    half = 0.5 if act == "silu" else 1.0
    gy, W = one_per_row(M, N, M), mantissas(K * N, N).view(K, N)
    x = torch.zeros(M, K)
    top = min(M, N)
    x[:top] = mantissas(top * K, 1).view(top, K)  # row j meets the one entry of gy in column j
    z = torch.zeros(M, N, device="cuda") if act == "silu" else None
    gx, gW, gx_alone = out(M, K, torch.float32), torch.full((K, N), float("nan"), device="cuda"), out(M, K, torch.float32)
    dense.etp_linear_vjp(x.cuda(), W.cuda(), gy.cuda(), z, ref.ACTS[act], gx, gW, None, workspace(M, K, N, torch.float32))
    dense.etp_linear_vjp(None, W.cuda(), gy.cuda(), z, ref.ACTS[act], gx_alone)
    d = half * gy.double().sum(1)
    want = d[:, None] * W.double().T[torch.arange(M) % N]
    check_products(gx, want, "grad_x")
    check_products(gx_alone, want, "grad_x alone")
    gw = torch.zeros(K, N, dtype=torch.float64)
    gw[:, :top] = x[:top].double().T * d[:top]
    check_products(gW, gw, "grad_W")


@pytest.mark.parametrize("K,N", [(64, 64), (200, 40), (200, 300)])
def test_largest_floats(K, N):
    """Floats above the largest bf16 (3.39e38) are split like the others."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("largest floats", K, N)
    M, top = 600, torch.finfo(torch.float32).max
    x = torch.zeros(M, K)
    r = torch.arange(M)
    x[r, r % K] = torch.where(r % 2 == 0, top, -3.396e38)
    W = (mantissas(K * N, 5).abs().view(K, N) * 2.0 ** -14)
    y = out(M, N, torch.float32)
    dense.etp_linear(x.cuda(), W.cuda(), y)
    check_products(y, x.double().sum(1, keepdim=True) * W.double()[r % K], "y")
    gW = torch.full((K, N), float("nan"), device="cuda")
    gy = one_per_row(M, N, 2) * 2.0 ** -14
    lead = min(M, N)
    x = torch.zeros(M, K)
    x[:lead] = top
    dense.etp_linear_vjp(x.cuda(), W.cuda(), gy.cuda(), None, 0, None, gW, None, workspace(M, K, N, torch.float32))
    gw = torch.zeros(K, N, dtype=torch.float64)
    gw[:, :lead] = x[:lead].double().T * gy[:lead].double().sum(1)
    check_products(gW, gw, "grad_W")


@pytest.mark.parametrize("r,c", [(1, 1), (24, 40), (128, 128), (60, 500), (200, 300), (300, 200)])
def test_scale_beyond_a_float(r, c):
    """1 / (|G|_F + eps) is not always a float: a zero matrix with an eps below 2^-128 stays zero, and entries near the
    largest float (a scale below the smallest normal float) give what the same matrix gives at any other scale."""
    import torch
    from test_gpu_dense_orth import make, run
    say("orth scale", r, c)
    for dtype in TYPES:
        zero = torch.zeros(2, r, c, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
        assert (run(zero, eps=1e-40) == 0).all()
        G = make(1, r, c, dtype, 4, scale=0.25)
        big = G * 2.0 ** 125  # exact
        assert torch.isfinite(big).all()
        assert torch.equal(run(big, eps=1e-30), run(G, eps=1e-40))
        small = G * 2.0 ** -120
        X = run(small, eps=1e-45)
        if dtype == "f32":  # (entries below the smallest normal float keep fewer bits)
            want = ref.orthogonalize(small, eps=1e-45)
            assert float((ref.f64(X) - want).norm()) <= 1.2e-4 * float(want.norm())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_between_the_tails(act):
    """Value and slope on a dense grid of [-6, 6]. SiLU: the logistic function errs by three units (2^-22 of it), its
    complement as a float by as much absolutely, times 1 + |z| in the slope. GELU: the fitted polynomial is within 8e-6
    of the tail (3.7e-9 of Phi), the float evaluation of its eight terms, the exponential of z^2 / 2 and 1 - tail add
    2^-21 of Phi and 2^-19 of the tail; the slope adds z times the density, an exponential of its own."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("activations", act)
    n = 120001
    z = torch.linspace(-6, 6, n)[:, None]
    one = torch.ones(1, 1, device="cuda")
    y, gx = out(n, 1, torch.float32), out(n, 1, torch.float32)
    dense.etp_linear(z.cuda(), one, y, None, ref.ACTS[act])
    dense.etp_linear_vjp(None, one, torch.ones_like(y), z.cuda(), ref.ACTS[act], gx)
    zd = z.double()
    if act == "silu":
        s = torch.sigmoid(zd)
        lim_y, lim_s = 2.0 ** -21 * s * zd.abs(), 2.0 ** -21 * s * (1 + zd.abs())
    else:
        tail = 0.5 * torch.erfc(zd.abs() / 2 ** 0.5)
        phi = torch.where(zd > 0, 1 - tail, tail)
        lim_phi = 2.0 ** -21 * phi + (8e-6 + 2.0 ** -19) * tail
        density = torch.exp(-zd * zd / 2) / (2 * torch.pi) ** 0.5
        lim_y = lim_phi * zd.abs() + 2.0 ** -23 * phi * zd.abs()
        lim_s = lim_phi + (2.0 ** -22 * (1 + zd * zd)) * zd.abs() * density + 2.0 ** -23
    for t, r, lim in ((y, ref.act(act, zd), lim_y), (gx, ref.act_slope(act, zd), lim_s)):
        err = (ref.f64(t) - r).abs()
        assert (err <= lim + 1e-30).all(), (float((err / (lim + 1e-30)).max()), float(zd[(err / (lim + 1e-30)).argmax()]))


@pytest.mark.parametrize("K,N", [(64, 64), (200, 40), (200, 300)])
def test_smallest_floats(K, N):
    """Below 2^-110 the last part is a subnormal bf16 of the unit 2^-133: half of that times the other factor."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("smallest floats", K, N)
    M = 600
    r = torch.arange(M)
    v = mantissas(M, 6)
    v = v / torch.exp2(torch.floor(torch.log2(v.abs()))) * torch.exp2(-(100 + r % 26).float())
    W = mantissas(K * N, 5).view(K, N)
    x, gy = torch.zeros(M, K), torch.zeros(M, N)
    x[r, r % K], gy[r, r % N] = v, v
    y, gx = out(M, N, torch.float32), out(M, K, torch.float32)
    dense.etp_linear(x.cuda(), W.cuda(), y)
    dense.etp_linear_vjp(None, W.cuda(), gy.cuda(), None, 0, gx)
    for got, w in ((y, W.double()[r % K]), (gx, W.double().T[r % N])):
        want = v.double()[:, None] * w
        err = (ref.f64(got) - want).abs()
        assert (err <= ONE_PRODUCT * want.abs() + 2.0 ** -134 * w.abs() + 2.0 ** -149).all()

"""GPU parity of the linear layer (etp_linear) and its VJP against float64:
every entry within 1e-5 of the largest one for float outputs (the bar of the
other fp32 calls; a float dot product of K <= 2048 random terms errs by about
sqrt(K) 2^-24 of its norm), plus half a bf16 unit where the output is bf16."""
import pytest

import dense_reference as ref

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1), (1, 64, 64), (2, 3, 5), (17, 8, 64), (63, 64, 1), (64, 1, 64), (65, 33, 31), (128, 128, 128),
          (200, 77, 201), (257, 256, 96), (130, 512, 40), (96, 40, 512), (1000, 64, 64), (70, 600, 700),
          (33, 1030, 17), (4100, 128, 64), (300, 160, 160), (520, 264, 392)]
TYPES = ["f32", "bf16"]


def say(*a):
    print("[case]", *a, flush=True)


def make(M, K, N, dtype, seed, pitch=0, zscale=1.0):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    rows = lambda n: rnd(M, n + pitch).to(dt).cuda()[:, :n]
    return dict(x=rows(K), W=(rnd(K, N) / K ** 0.5).to(dt).cuda(), b=rnd(N).cuda(), res=rows(N),
                z=(rnd(M, N + pitch) * zscale).to(dt).cuda()[:, :N], gy=rows(N), dt=dt)


def out(M, N, dt, pitch=0, fill=float("nan")):
    import torch
    return torch.full((M, N + pitch), fill, dtype=dt, device="cuda")[:, :N]


def workspace(M, K, N, dt):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    return torch.full((max(16, dense.etp_linear_vjp_workspace(M, K, N, dt)),), 0xFF, dtype=torch.uint8, device="cuda")


def run_vjp(p, act, M, K, N, pitch=0, flags=0, base=None, **kw):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    gx = out(M, K, p["dt"], pitch) if base is None else base[0]
    gW = torch.full((K, N), float("nan"), device="cuda") if base is None else base[1]
    gb = torch.full((N,), float("nan"), device="cuda") if base is None else base[2]
    dense.etp_linear_vjp(p["x"], p["W"], p["gy"], p["z"] if act != "none" else None, ref.ACTS[act], gx, gW, gb,
                         workspace(M, K, N, p["dt"]), flags, **kw)
    return gx, gW, gb


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward(M, K, N, dtype):
    from equivariant_interatomic_potentials_amd import dense
    act = ["none", "silu", "gelu"][(M + K + N) % 3]
    say("linear", M, K, N, dtype, act)
    p = make(M, K, N, dtype, M + 7 * K + 13 * N)
    y, z = out(M, N, p["dt"]), out(M, N, p["dt"])
    dense.etp_linear(p["x"], p["W"], y, p["b"], ref.ACTS[act], p["res"], z)
    yr, zr = ref.linear(p["x"], p["W"], p["b"], act, p["res"])
    ref.close(y, yr)
    ref.close(z, zr)
    y2 = out(M, N, p["dt"])
    dense.etp_linear(p["x"], p["W"], y2)  # no bias, activation, residual or z
    ref.close(y2, ref.linear(p["x"], p["W"])[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_vjp(M, K, N, dtype):
    act = ["silu", "gelu", "none"][(M + K + N) % 3]
    say("linear_vjp", M, K, N, dtype, act)
    p = make(M, K, N, dtype, 3 * M + 7 * K + N)
    got = run_vjp(p, act, M, K, N)
    for g, r in zip(got, ref.linear_vjp(p["x"], p["W"], p["gy"], p["z"], act)):
        ref.close(g, r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("pitch", [1, 8])
@pytest.mark.parametrize("K,N", [(64, 64), (40, 72), (264, 392)])
def test_strided_rows_leave_the_gaps(act, dtype, pitch, K, N):
    """Rows longer than the matrix: the entries between them are neither read (NaN in the inputs) nor written."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    M = 150
    say("linear strided", K, N, dtype, act, pitch)
    p = make(M, K, N, dtype, 5, pitch)
    for k in ("x", "res", "z", "gy"):
        p[k]._base[:, p[k].shape[1]:] = float("nan")
    y, z = out(M, N, p["dt"], pitch, 7.0), out(M, N, p["dt"], pitch, 7.0)
    dense.etp_linear(p["x"], p["W"], y, p["b"], ref.ACTS[act], p["res"], z)
    yr, zr = ref.linear(p["x"], p["W"], p["b"], act, p["res"])
    ref.close(y, yr)
    ref.close(z, zr)
    gx = out(M, K, p["dt"], pitch, 7.0)
    base = (gx, torch.empty(K, N, device="cuda"), torch.empty(N, device="cuda"))
    for g, r in zip(run_vjp(p, act, M, K, N, base=base), ref.linear_vjp(p["x"], p["W"], p["gy"], p["z"], act)):
        ref.close(g, r)
    for t in (y, z, gx):
        assert (t._base[:, t.shape[1]:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_misaligned_bases(dtype):
    """Views that start one element into their storage."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    M, K, N = 130, 64, 64
    say("linear misaligned", dtype)
    p = make(M, K, N, dtype, 8)

    def shift(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        s.copy_(t)
        return s

    p.update({k: shift(p[k]) for k in ("x", "W", "b", "res", "z", "gy")})
    y, z = shift(out(M, N, p["dt"])), shift(out(M, N, p["dt"]))
    dense.etp_linear(p["x"], p["W"], y, p["b"], 1, p["res"], z)
    yr, zr = ref.linear(p["x"], p["W"], p["b"], "silu", p["res"])
    ref.close(y, yr)
    ref.close(z, zr)
    base = (shift(out(M, K, p["dt"])), shift(torch.empty(K, N, device="cuda")), shift(torch.empty(N, device="cuda")))
    for g, r in zip(run_vjp(p, "silu", M, K, N, base=base), ref.linear_vjp(p["x"], p["W"], p["gy"], p["z"], "silu")):
        ref.close(g, r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(70, 64, 64), (50, 130, 300), (3000, 128, 96)])
def test_vjp_accumulates(M, K, N, dtype):
    import torch
    from equivariant_interatomic_potentials_amd import etp
    say("linear_vjp accumulate", M, K, N, dtype)
    p = make(M, K, N, dtype, 9)
    g = torch.Generator().manual_seed(2)
    base = (torch.randn(M, K, generator=g).to(p["dt"]).cuda(), torch.randn(K, N, generator=g).cuda(),
            torch.randn(N, generator=g).cuda())
    was = [ref.f64(t) for t in base]
    got = run_vjp(p, "silu", M, K, N, flags=etp.ETP_FLAG_ACCUMULATE, base=base)
    for t, b, r in zip(got, was, ref.linear_vjp(p["x"], p["W"], p["gy"], p["z"], "silu")):
        ref.close(t, b + r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(200, 64, 64), (90, 300, 130)])
def test_vjp_outputs_are_optional(M, K, N, dtype):
    """Each output alone equals the same output of the full call bit for bit or within the bar."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("linear_vjp optional", M, K, N, dtype)
    p = make(M, K, N, dtype, 10)
    want = ref.linear_vjp(p["x"], p["W"], p["gy"], p["z"], "gelu")
    for which in range(3):
        o = [None, None, None]
        o[which] = [out(M, K, p["dt"]), torch.empty(K, N, device="cuda"), torch.empty(N, device="cuda")][which]
        dense.etp_linear_vjp(p["x"] if which == 1 else None, p["W"], p["gy"], p["z"], 2, *o,
                             workspace(M, K, N, p["dt"]) if which else None)
        ref.close(o[which], want[which])


@pytest.mark.parametrize("dtype", TYPES)
def test_no_rows(dtype):
    import torch
    from equivariant_interatomic_potentials_amd import dense, etp
    K, N = 20, 30
    say("linear no rows", dtype)
    p = make(0, K, N, dtype, 1)
    y = out(0, N, p["dt"])
    dense.etp_linear(p["x"], p["W"], y, p["b"], 1)
    gx, gW, gb = run_vjp(p, "silu", 0, K, N)
    assert (gW == 0).all() and (gb == 0).all()
    gW.fill_(2.0)
    gb.fill_(3.0)
    dense.etp_linear_vjp(p["x"], p["W"], p["gy"], p["z"], 1, None, gW, gb, None, etp.ETP_FLAG_ACCUMULATE)
    assert (gW == 2).all() and (gb == 3).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_saturated_activations(act, dtype):
    """Pre-activations far into both tails: value and slope stay finite and right."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("linear saturated", act, dtype)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    v = torch.tensor([-3e38, -1e30, -1e4, -200., -100., -88., -40., -8., -1e-3, -1e-30, 0., 1e-30, 1e-3, 8., 40., 88.,
                      100., 200., 1e4, 1e30, 3e38], dtype=dt)
    x = v[:, None].cuda()
    one = torch.ones(1, 1, dtype=dt, device="cuda")
    y, z = out(len(v), 1, dt), out(len(v), 1, dt)
    dense.etp_linear(x, one, y, None, ref.ACTS[act], None, z)
    yr = ref.act(act, v.double()[:, None])
    assert torch.equal(z.cpu(), v[:, None])
    small = yr.abs() < 1e10
    ref.close(torch.where(small.cuda(), y, torch.zeros_like(y)), torch.where(small, yr, 0 * yr), scale=1.0)
    big = ~small
    assert ((ref.f64(y) - yr).abs()[big] <= yr.abs()[big] * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22)).all()
    gx, gW, gb = out(len(v), 1, dt), torch.empty(1, 1, device="cuda"), torch.empty(1, device="cuda")
    dense.etp_linear_vjp(x, one, torch.ones_like(y), z, ref.ACTS[act], gx, None, gb,
                         workspace(len(v), 1, 1, dt))
    sr = ref.act_slope(act, v.double()[:, None])
    ref.close(gx, sr, scale=2.0)
    ref.close(gb, sr.sum(0), scale=20.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K,N", [(64, 64), (200, 300)])
def test_nan_and_infinity_stay_in_their_row(K, N, dtype):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    M = 100
    say("linear non-finite", K, N, dtype)
    p = make(M, K, N, dtype, 4)
    clean = out(M, N, p["dt"])
    dense.etp_linear(p["x"], p["W"], clean, p["b"], 1)
    p["x"][3, 5] = float("nan")
    p["x"][70, 0] = float("inf")
    y = out(M, N, p["dt"], fill=0.0)
    dense.etp_linear(p["x"], p["W"], y, p["b"], 0)
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[70]).any()
    dense.etp_linear(p["x"], p["W"], y, p["b"], 1)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[3, 70]] = False
    assert torch.equal(y[keep], clean[keep])
    gx0 = run_vjp(p, "silu", M, K, N)[0].clone()
    p["gy"][9, 1] = float("nan")
    gx, gW, gb = run_vjp(p, "silu", M, K, N)
    keep = torch.arange(M, device="cuda") != 9
    assert torch.isnan(gx[9]).all() and torch.equal(gx[keep], gx0[keep])
    assert torch.isnan(gb[1]) and torch.isfinite(gb[[0, 2]]).all() and torch.isnan(gW[:, 1]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_offsets_beyond_32_bits(dtype):
    """A row pitch that puts the last rows past 2^31 elements: input, output and gradient in place."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    M, K, N, pitch = 66000, 64, 32, 33000
    say("linear offsets", dtype)
    big = torch.empty(M, pitch, dtype=dt, device="cuda")
    x, y, gx = big[:, :K], big[:, 1000:1000 + N], big[:, 20000:20000 + K]
    g = torch.Generator(device="cuda").manual_seed(3)
    x.copy_(torch.randn(M, K, generator=g, device="cuda"))
    W = (torch.randn(K, N, generator=g, device="cuda") / 8).to(dt)
    gy = torch.randn(M, N, generator=g, device="cuda").to(dt)
    dense.etp_linear(x, W, y)
    gW = torch.empty(K, N, device="cuda")
    dense.etp_linear_vjp(x, W, gy, None, 0, gx, gW, None, workspace(M, K, N, dt))
    last = slice(M - 200, M)
    ref.close(y[last], ref.linear(x[last], W)[0])
    ref.close(gx[last], ref.f64(gy[last]) @ ref.f64(W).T)
    ref.close(gW, (x.double().T.contiguous() @ gy.double()).cpu())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(5000, 64, 64), (700, 300, 200)])
def test_bitwise_repeatable_and_on_a_stream(M, K, N, dtype):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("linear repeat", M, K, N, dtype)
    p = make(M, K, N, dtype, 21)
    y = out(M, N, p["dt"])
    dense.etp_linear(p["x"], p["W"], y, p["b"], 1)
    first = (y.clone(), *[t.clone() for t in run_vjp(p, "silu", M, K, N)])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2 = out(M, N, p["dt"])
    base = (out(M, K, p["dt"]), torch.empty(K, N, device="cuda"), torch.empty(N, device="cuda"))
    ws = workspace(M, K, N, p["dt"])
    torch.cuda.synchronize()
    dense.etp_linear(p["x"], p["W"], y2, p["b"], 1, stream=s)
    dense.etp_linear_vjp(p["x"], p["W"], p["gy"], p["z"], 1, *base, ws, stream=s)
    s.synchronize()
    for a, b in zip(first, (y2, *base)):
        assert torch.equal(a, b)


def test_vjp_against_differences():
    """<gx, v> + <gW, V> + <gb, u> is the slope of <gy, y> along (v, V, u): central differences of the forward, step
    2^-6 (truncation of order step^2 times third derivatives, rounding of order 2^-24 / step)."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    M, K, N, h = 40, 24, 36, 2.0 ** -6
    for act in ("silu", "gelu"):
        say("linear differences", act)
        p = make(M, K, N, "f32", 31)
        g = torch.Generator().manual_seed(5)
        v, V, u = (torch.randn(*s, generator=g).cuda() for s in ((M, K), (K, N), (N,)))

        def f(t):
            y = out(M, N, torch.float32)
            dense.etp_linear(p["x"] + t * v, p["W"] + t * V, y, p["b"] + t * u, ref.ACTS[act], p["res"])
            return float((y.double() * p["gy"].double()).sum())

        y = out(M, N, torch.float32)
        dense.etp_linear(p["x"], p["W"], y, p["b"], ref.ACTS[act], p["res"], p["z"])
        gx, gW, gb = run_vjp(p, act, M, K, N)
        slope = sum(float((a.double() * b.double()).sum()) for a, b in ((gx, v), (gW, V), (gb, u)))
        # fourth-order: Richardson on steps h and h / 2
        d1, d2 = (f(h) - f(-h)) / (2 * h), (f(h / 2) - f(-h / 2)) / h
        size = sum(float((a.double() * b.double()).square().sum()) ** 0.5 for a, b in ((gx, v), (gW, V), (gb, u)))
        assert abs((4 * d2 - d1) / 3 - slope) < 1e-3 * size, (d1, d2, slope, size)

"""GPU parity of the grouped layer (etp_grouped_linear) and its VJP against
float64, group by group, with the bars of the ungrouped layer: every entry within
1e-5 of the largest one for float outputs (a float dot product of K <= 2048 random
terms errs by about sqrt(K) 2^-24 of its norm), plus half a bf16 unit where the
output is bf16. In the gradients, where few entries may all be sums that cancel,
the largest norm of an entry's terms counts where it is larger
(grouped_reference.linear_vjp_terms says why)."""
import pytest

import dense_reference as ref
import grouped_reference as gref

pytestmark = pytest.mark.gpu

# rows, groups, n_in, n_out
SHAPES = [(1, 1, 1, 1), (1, 5, 64, 64), (2, 3, 3, 5), (17, 4, 8, 64), (63, 1, 64, 1), (64, 64, 1, 64), (65, 2, 33, 31),
          (21, 64, 128, 128), (200, 3, 77, 201), (257, 9, 256, 96), (130, 2, 512, 40), (96, 30, 40, 512),
          (1000, 25, 64, 64), (70, 7, 600, 700), (33, 2, 1030, 17), (4100, 16, 128, 64), (300, 3, 160, 160),
          (520, 5, 264, 392), (3000, 2000, 24, 40), (6000, 10, 300, 64), (9000, 4, 256, 30), (5000, 3, 130, 260)]
TYPES = ["f32", "bf16"]


def say(*a):
    print("[case]", *a, flush=True)


def make(M, G, K, N, dtype, seed, pitch=0, order=True, pad=0.1, zscale=1.0):
    """Rows in uneven groups (a tenth in none), features, and everything the calls take."""
    import numpy as np
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    rows = lambda n: rnd(M, n + pitch).to(dt).cuda()[:, :n]
    ids = (torch.rand(M, generator=g).double() ** 2 * G).long().clamp_(max=G - 1)
    if pad and M > 1:
        ids[torch.rand(M, generator=g) < pad] = -1
    if not order:
        ids = torch.sort(torch.where(ids < 0, G, ids)).values
    ptr, o = gref.group_rows(ids.numpy(), G)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return dict(x=rows(K), W=(rnd(G, K, N) / K ** 0.5).to(dt).cuda(), b=rnd(G, N).cuda(), res=rows(N),
                z=(rnd(M, N + pitch) * zscale).to(dt).cuda()[:, :N], gy=rows(N), dt=dt, ptr=cuda(ptr),
                order=cuda(o) if order else None, G=G)


def out(M, N, dt, pitch=0, fill=7.0):
    import torch
    return torch.full((M, N + pitch), fill, dtype=dt, device="cuda")[:, :N]


def workspace(M, G, K, N, dt):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    size = dense.etp_grouped_linear_vjp_workspace(M, G, K, N, dt)
    return torch.full((max(16, size),), 0xFF, dtype=torch.uint8, device="cuda")


def run_fwd(p, act, M, N, pitch=0, **kw):
    from equivariant_interatomic_potentials_amd import dense
    y, z = out(M, N, p["dt"], pitch), out(M, N, p["dt"], pitch)
    dense.etp_grouped_linear(p["x"], p["W"], y, p["ptr"], p["order"], p["b"], ref.ACTS[act], p["res"], z, **kw)
    return y, z


def want_fwd(p, act, y0, z0):
    return gref.linear(p["x"], p["W"], p["ptr"], p["order"], p["b"], act, p["res"], y0, z0)


def run_vjp(p, act, M, K, N, pitch=0, flags=0, base=None, **kw):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    G = p["G"]
    base = base or (out(M, K, p["dt"], pitch), torch.full((G, K, N), float("nan"), device="cuda"),
                    torch.full((G, N), float("nan"), device="cuda"))
    dense.etp_grouped_linear_vjp(p["x"], p["W"], p["gy"], p["ptr"], p["order"], p["z"] if act != "none" else None,
                                 ref.ACTS[act], *base, workspace(M, G, K, N, p["dt"]), flags, **kw)
    return base


def want_vjp(p, act, gx0):
    return gref.linear_vjp(p["x"], p["W"], p["gy"], p["ptr"], p["order"], p["z"], act, gx0)


def close_vjp(got, p, act, gx0):
    terms = gref.linear_vjp_terms(p["x"], p["W"], p["gy"], p["ptr"], p["order"], p["z"], act)
    for g, r, t in zip(got, want_vjp(p, act, gx0), terms):
        ref.close(g, r, scale=max(t, float(r.abs().max()) if r.numel() else 0.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,G,K,N", SHAPES)
def test_forward(M, G, K, N, dtype):
    from equivariant_interatomic_potentials_amd import dense
    act = ["none", "silu", "gelu"][(M + K + N) % 3]
    say("grouped", M, G, K, N, dtype, act)
    for order in (True, False):
        p = make(M, G, K, N, dtype, M + 7 * K + 13 * N, order=order)
        y0 = out(M, N, p["dt"])
        y, z = run_fwd(p, act, M, N)
        yr, zr = want_fwd(p, act, y0, y0)
        ref.close(y, yr)
        ref.close(z, zr)
        y2 = out(M, N, p["dt"])
        dense.etp_grouped_linear(p["x"], p["W"], y2, p["ptr"], p["order"])  # no bias, activation, residual or z
        ref.close(y2, gref.linear(p["x"], p["W"], p["ptr"], p["order"], y0=y0)[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,G,K,N", SHAPES)
def test_vjp(M, G, K, N, dtype):
    say("grouped vjp", M, G, K, N, dtype)
    for act in (["silu", "gelu"][(M + K + N) % 2], "none"):
        for order in (True, False):
            p = make(M, G, K, N, dtype, 3 * M + 7 * K + N, order=order)
            close_vjp(run_vjp(p, act, M, K, N), p, act, out(M, K, p["dt"]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("pitch", [1, 8])
@pytest.mark.parametrize("M,K,N", [(150, 64, 64), (150, 40, 72), (150, 264, 392), (9000, 264, 136), (9000, 72, 96)])
def test_strided_rows_and_rows_in_no_group(M, K, N, act, pitch, dtype):
    """What lies between the rows, and rows in no group, are neither read (NaN in the inputs) nor written."""
    import torch
    say("grouped strided", M, K, N, dtype, act, pitch)
    p = make(M, 6, K, N, dtype, 5, pitch, pad=0.3)
    free = p["order"][int(p["ptr"][-1]):].long()
    assert len(free) > 5
    for k in ("x", "res", "z", "gy"):
        p[k]._base[:, p[k].shape[1]:] = float("nan")
        p[k][free] = float("nan")
    y, z = run_fwd(p, act, M, N, pitch)
    o7 = out(M, N, p["dt"])
    yr, zr = want_fwd(p, act, o7, o7)
    ref.close(y, yr)
    ref.close(z, zr)
    gx, gW, gb = run_vjp(p, act, M, K, N, pitch)
    for g, r in zip((gx, gW, gb), want_vjp(p, act, out(M, K, p["dt"]))):
        ref.close(g, r)
    for t in (y, z, gx):
        assert (t._base[:, t.shape[1]:] == 7.0).all() and (t[free] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes", [[0, 0, 5], [64, 0, 0, 64], [1] * 40, [0] * 70 + [3] + [0] * 70, [129, 1, 127],
                                   [0], [33, 0, 2000, 1, 0], [63, 65, 64, 128, 16, 15, 17, 1]])
@pytest.mark.parametrize("K,N", [(64, 48), (200, 150)])
def test_group_boundaries(sizes, K, N, dtype):
    """Sizes at and next to the tiles', empty groups first, last and in runs; slots before the first group and behind
    the last are left alone."""
    import torch
    G, before, behind = len(sizes), 5, 9
    M = before + sum(sizes) + behind
    say("grouped boundaries", sizes[:6], G, K, N, dtype)
    p = make(M, G, K, N, dtype, 11, order=True)
    p["ptr"] = (before + torch.cat([torch.zeros(1), torch.tensor(sizes).cumsum(0)])).to(torch.int32).cuda()
    for order in (p["order"], None):
        p["order"] = order
        o7 = out(M, N, p["dt"])
        y, z = run_fwd(p, "silu", M, N)
        for g, r in zip((y, z), want_fwd(p, "silu", o7, o7)):
            ref.close(g, r)
        for act in ("gelu", "none"):
            close_vjp(run_vjp(p, act, M, K, N), p, act, out(M, K, p["dt"]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 700, 9000])
@pytest.mark.parametrize("K,N", [(64, 48), (200, 150)])
def test_long_runs_of_empty_groups(rows, K, N, dtype):
    """Groups with rows behind 62, 63, 64, 65 and 500 empty ones: one run of tiles meets several, or ends in one."""
    import numpy as np
    import torch
    say("empty runs", rows, K, N, dtype)
    sizes = [5] + [0] * 62 + [129] + [0] * 63 + [rows] + [0] * 64 + [3] + [0] * 65 + [rows] + [0] * 500 + [2, 0, 1] + [0] * 130
    M, G = sum(sizes), len(sizes)
    p = make(M, G, K, N, dtype, rows + K)
    ptr = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    p.update(ptr=ptr, order=torch.randperm(M, generator=torch.Generator().manual_seed(3)).int().cuda())
    y, z = run_fwd(p, "silu", M, N)
    o7 = out(M, N, p["dt"])
    for g, r in zip((y, z), want_fwd(p, "silu", o7, o7)):
        ref.close(g, r)
    close_vjp(run_vjp(p, "silu", M, K, N), p, "silu", out(M, K, p["dt"]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,G,K,N", [(70001, 4, 64, 64), (70001, 40, 64, 128), (40000, 3, 128, 30), (50000, 100, 20, 96),
                                     (33000, 5, 300, 128), (20000, 64, 256, 256), (30000, 2, 136, 512),
                                     (12000, 1, 512, 136), (60000, 700, 48, 33)])
def test_many_rows(M, G, K, N, dtype):
    """Row counts that fill the chip several times over: groups that cross workgroups' runs, and many within one."""
    act = ["silu", "gelu", "none"][(M + G + K) % 3]
    say("grouped many", M, G, K, N, dtype, act)
    p = make(M, G, K, N, dtype, M + K)
    o7 = out(M, N, p["dt"])
    for g, r in zip(run_fwd(p, act, M, N), want_fwd(p, act, o7, o7)):
        ref.close(g, r)
    for g, r in zip(run_vjp(p, act, M, K, N), want_vjp(p, act, out(M, K, p["dt"]))):
        ref.close(g, r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,G,K,N", [(70, 3, 64, 64), (50, 2, 130, 300), (3000, 12, 128, 96), (4000, 70, 200, 40)])
def test_vjp_accumulates(M, G, K, N, dtype):
    import torch
    from equivariant_interatomic_potentials_amd import etp
    say("grouped accumulate", M, G, K, N, dtype)
    for act in ("silu", "none"):
        p = make(M, G, K, N, dtype, 9)
        g = torch.Generator().manual_seed(2)
        base = (torch.randn(M, K, generator=g).to(p["dt"]).cuda(), torch.randn(G, K, N, generator=g).cuda(),
                torch.randn(G, N, generator=g).cuda())
        was = [ref.f64(t) for t in base]
        got = run_vjp(p, act, M, K, N, flags=etp.ETP_FLAG_ACCUMULATE, base=base)
        wx, wW, wb = want_vjp(p, act, torch.zeros(M, K))
        for t, b, r in zip(got, was, (wx, wW, wb)):
            ref.close(t, b + r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,G,K,N", [(0, 3, 6, 7), (300, 4, 64, 64), (700, 3, 200, 50), (700, 8, 50, 200),
                                     (900, 5, 260, 300)])
def test_every_subset_of_the_gradients(M, G, K, N, dtype):
    """The workspace holds what any subset needs, and what is not asked for is not written."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("grouped subsets", M, G, K, N, dtype)
    p = make(M, G, K, N, dtype, M + K)
    for act in ("gelu", "none"):
        want = want_vjp(p, act, out(M, K, p["dt"]))
        for which in range(1, 8):
            new = [out(M, K, p["dt"]), torch.full((G, K, N), float("nan"), device="cuda"),
                   torch.full((G, N), float("nan"), device="cuda")]
            o = [t if which >> i & 1 else None for i, t in enumerate(new)]
            size = dense.etp_grouped_linear_vjp_workspace(M, G, K, N, p["dt"])
            ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
            dense.etp_grouped_linear_vjp(p["x"] if which & 2 else None, p["W"] if which & 1 else None, p["gy"], p["ptr"],
                                         p["order"], p["z"], ref.ACTS[act], *o, ws[:size] if size else None)
            assert (ws[size:] == 0xFF).all()
            for t, r in zip(o, want):
                if t is not None:
                    ref.close(t, r)


@pytest.mark.parametrize("dtype", TYPES)
def test_misaligned_bases(dtype):
    """Views that start one element into their storage."""
    import torch
    M, G, K, N = 130, 3, 64, 64
    say("grouped misaligned", dtype)
    p = make(M, G, K, N, dtype, 8)

    def shift(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        s.copy_(t)
        return s

    p.update({k: shift(p[k]) for k in ("x", "W", "b", "res", "z", "gy", "ptr", "order")})
    o7 = out(M, N, p["dt"])
    for g, r in zip(run_fwd(p, "silu", M, N), want_fwd(p, "silu", o7, o7)):
        ref.close(g, r)
    base = (shift(out(M, K, p["dt"])), shift(torch.empty(G, K, N, device="cuda")), shift(torch.empty(G, N, device="cuda")))
    for act in ("silu", "none"):
        for g, r in zip(run_vjp(p, act, M, K, N, base=base), want_vjp(p, act, out(M, K, p["dt"]))):
            ref.close(g, r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K,N", [(64, 64), (200, 300)])
def test_nan_and_infinity_stay_in_their_row_and_group(K, N, dtype):
    import torch
    M, G = 400, 4
    say("grouped non-finite", K, N, dtype)
    p = make(M, G, K, N, dtype, 4, pad=0)
    clean = run_fwd(p, "silu", M, N)[0]
    gx0, gW0, gb0 = (t.clone() for t in run_vjp(p, "silu", M, K, N))
    row = int(p["order"][int(p["ptr"][2])])  # the first row of group 2
    x = p["x"].clone()
    p["x"][row, 5] = float("nan")
    y = run_fwd(p, "silu", M, N)[0]
    keep = torch.arange(M, device="cuda") != row
    assert torch.isnan(y[row]).all() and torch.equal(y[keep], clean[keep])
    p["x"].copy_(x)
    p["gy"][row, 1] = float("nan")
    gx, gW, gb = run_vjp(p, "silu", M, K, N)
    assert torch.isnan(gx[row]).all() and torch.equal(gx[keep], gx0[keep])
    other = torch.tensor([0, 1, 3], device="cuda")
    assert torch.equal(gW[other], gW0[other]) and torch.equal(gb[other], gb0[other])
    assert torch.isnan(gb[2, 1]) and torch.isfinite(gb[2, 2:]).all() and torch.isnan(gW[2, :, 1]).all()
    p["gy"][row, 1] = 0.0
    p["W"][1] = float("nan")  # another group's matrix
    y = run_fwd(p, "silu", M, N)[0]
    mine = p["order"][int(p["ptr"][1]):int(p["ptr"][2])].long()
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[mine] = False
    assert torch.isnan(y[mine]).all() and torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("dtype", TYPES)
def test_indexes_that_are_no_rows_are_passed_over(dtype):
    """Offsets outside the rows are held to them and indexes outside are skipped: nothing else is read or written."""
    import torch
    M, G, K, N = 200, 3, 40, 24
    say("grouped bad indexes", dtype)
    p = make(M, G, K, N, dtype, 6, pad=0)
    want, _ = want_fwd(p, "none", out(M, N, p["dt"]), out(M, N, p["dt"]))
    bad = torch.tensor([3, 50, 199], device="cuda")
    gone = p["order"][bad].long()
    p["order"][bad] = torch.tensor([-1, M, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    p["ptr"][0], p["ptr"][-1] = -17, 2 ** 31 - 1
    y, _ = run_fwd(p, "none", M, N)
    want[gone.cpu()] = 7.0
    ref.close(y, want)
    gx, gW, gb = run_vjp(p, "none", M, K, N)
    keep = torch.ones(M, 1, device="cuda")
    keep[gone] = 0
    p["gy"].mul_(keep.to(p["dt"]))
    p["order"][bad] = gone.to(torch.int32)
    p["ptr"][0], p["ptr"][-1] = 0, M
    wx, wW, wb = want_vjp(p, "none", out(M, K, p["dt"]))
    wx[gone.cpu()] = 7.0
    for g, r in zip((gx, gW, gb), (wx, wW, wb)):
        ref.close(g, r)


@pytest.mark.parametrize("dtype", TYPES)
def test_offsets_beyond_32_bits(dtype):
    """A row pitch that puts the last rows past 2^31 elements: input, output and gradient in place; then matrices whose
    last group lies past 2^31 elements."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    M, K, N, pitch = 66000, 64, 32, 33000
    say("grouped offsets", dtype)
    big = torch.empty(M, pitch, dtype=dt, device="cuda")
    x, y, gx = big[:, :K], big[:, 1000:1000 + N], big[:, 20000:20000 + K]
    g = torch.Generator(device="cuda").manual_seed(3)
    x.copy_(torch.randn(M, K, generator=g, device="cuda"))
    W = (torch.randn(2, K, N, generator=g, device="cuda") / 8).to(dt)
    gy = torch.randn(M, N, generator=g, device="cuda").to(dt)
    ptr = torch.tensor([0, 1000, M], dtype=torch.int32, device="cuda")
    order = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
    dense.etp_grouped_linear(x, W, y, ptr, order)
    gW = torch.empty(2, K, N, device="cuda")
    dense.etp_grouped_linear_vjp(x, W, gy, ptr, order, None, 0, gx, gW, None, workspace(M, 2, K, N, dt))
    last = slice(M - 200, M)  # the first slots: group 0
    ref.close(y[last], ref.linear(x[last], W[0])[0])
    ref.close(gx[last], ref.f64(gy[last]) @ ref.f64(W[0]).T)
    ref.close(gW[0], (x[M - 1000:].double().T.contiguous() @ gy[M - 1000:].double()).cpu())
    del big, x, y, gx
    G, K, N = 2300, 1024, 1024
    W = torch.zeros(G, K, N, dtype=dt, device="cuda")
    W[G - 1] = (torch.randn(K, N, generator=g, device="cuda") / 32).to(dt)
    x = torch.randn(20, K, generator=g, device="cuda").to(dt)
    gy = torch.randn(20, N, generator=g, device="cuda").to(dt)
    ptr = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    ptr[G - 1:] = torch.tensor([4, 20], dtype=torch.int32)
    ptr[1:G - 1] = 4
    y, gx = torch.empty(20, N, dtype=dt, device="cuda"), torch.empty(20, K, dtype=dt, device="cuda")
    gW = torch.full((G, K, N), float("nan"), device="cuda")
    dense.etp_grouped_linear(x, W, y, ptr)
    dense.etp_grouped_linear_vjp(x, W, gy, ptr, None, None, 0, gx, gW, None, workspace(20, G, K, N, dt))
    ref.close(y[4:], ref.linear(x[4:], W[G - 1])[0])
    assert (y[:4] == 0).all() and (gx[:4] == 0).all()
    ref.close(gx[4:], ref.f64(gy[4:]) @ ref.f64(W[G - 1]).T)
    ref.close(gW[G - 1], ref.f64(x[4:]).T @ ref.f64(gy[4:]))
    ref.close(gW[0], ref.f64(x[:4]).T @ ref.f64(gy[:4]))
    assert (gW[1:G - 1] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,G,K,N", [(5000, 7, 64, 64), (9000, 3, 300, 200), (21, 64, 128, 128)])
def test_bitwise_repeatable_on_a_stream_and_from_a_graph(M, G, K, N, dtype):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("grouped repeat", M, G, K, N, dtype)
    p = make(M, G, K, N, dtype, 21)
    first = [t.clone() for t in (*run_fwd(p, "silu", M, N), *run_vjp(p, "silu", M, K, N))]
    torch.cuda.synchronize()
    y, z = out(M, N, p["dt"]), out(M, N, p["dt"])
    base = (out(M, K, p["dt"]), torch.empty(G, K, N, device="cuda"), torch.empty(G, N, device="cuda"))
    ws = workspace(M, G, K, N, p["dt"])

    def calls(stream=None):
        dense.etp_grouped_linear(p["x"], p["W"], y, p["ptr"], p["order"], p["b"], 1, p["res"], z, stream=stream)
        dense.etp_grouped_linear_vjp(p["x"], p["W"], p["gy"], p["ptr"], p["order"], p["z"], 1, *base, ws, stream=stream)

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    calls(s)
    s.synchronize()
    for a, b in zip(first, (y, z, *base)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in range(3):
        p["x"].mul_(1.25)
        calls()
        want = [t.clone() for t in (y, z, *base)]
        for t in (y, z, *base):
            t.fill_(7.0)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (y, z, *base)):
            assert torch.equal(a, b), k


def test_vjp_against_differences():
    """<gx, v> + <gW, V> + <gb, u> is the slope of <gy, y> along (v, V, u): central differences of the forward at 2^-6
    and its half, extrapolated (truncation of order step^4, rounding of order 2^-24 / step)."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    M, G, K, N, h = 40, 3, 24, 36, 2.0 ** -6
    for act in ("silu", "gelu"):
        say("grouped differences", act)
        p = make(M, G, K, N, "f32", 31, pad=0)
        g = torch.Generator().manual_seed(5)
        v, V, u = (torch.randn(*s, generator=g).cuda() for s in ((M, K), (G, K, N), (G, N)))

        def f(t):
            y = out(M, N, torch.float32)
            dense.etp_grouped_linear(p["x"] + t * v, p["W"] + t * V, y, p["ptr"], p["order"], p["b"] + t * u,
                                     ref.ACTS[act], p["res"])
            return float((y.double() * p["gy"].double()).sum())

        p["z"] = run_fwd(p, act, M, N)[1]
        gx, gW, gb = run_vjp(p, act, M, K, N)
        slope = sum(float((a.double() * b.double()).sum()) for a, b in ((gx, v), (gW, V), (gb, u)))
        d1, d2 = (f(h) - f(-h)) / (2 * h), (f(h / 2) - f(-h / 2)) / h
        size = sum(float((a.double() * b.double()).square().sum()) ** 0.5 for a, b in ((gx, v), (gW, V), (gb, u)))
        assert abs((4 * d2 - d1) / 3 - slope) < 1e-3 * size, (d1, d2, slope, size)


def test_orientation_is_checked():
    import torch
    from equivariant_interatomic_potentials_amd import dense
    M, G, K, N = 30, 2, 40, 72
    say("grouped shapes")
    p = make(M, G, K, N, "f32", 3)
    ws = workspace(M, G, K, N, p["dt"])
    for gW in (torch.empty(G, N, K, device="cuda"), torch.empty(K, N, device="cuda")):
        with pytest.raises(ValueError, match="grad_W"):
            dense.etp_grouped_linear_vjp(p["x"], p["W"], p["gy"], p["ptr"], p["order"], p["z"], 1, None, gW, None, ws)
    with pytest.raises(ValueError, match="W must"):
        dense.etp_grouped_linear(p["x"], p["W"][:1], out(M, N, p["dt"]), p["ptr"], p["order"])
    with pytest.raises(ValueError, match="order"):
        dense.etp_grouped_linear(p["x"], p["W"], out(M, N, p["dt"]), p["ptr"], p["order"][1:])
    with pytest.raises(ValueError, match="bias"):
        dense.etp_grouped_linear(p["x"], p["W"], out(M, N, p["dt"]), p["ptr"], p["order"], p["b"][0])
    with pytest.raises(ValueError, match="device"):
        dense.etp_grouped_linear(p["x"], p["W"], out(M, N, p["dt"]), p["ptr"].cpu(), p["order"])

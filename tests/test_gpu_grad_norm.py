"""GPU parity of etp_grad_norm and etp_clip_grads. The norm is a double rounded
once to float: within 2^-24 of the float64 norm (and the summation's 2^-50 or
so, which 2^-40 covers). A
clipped float is the product with a double scale rounded once: half a step
of the result, 2^-24 relative, plus the scale's own rounding; a bf16 one is formed in
float from a float scale (2^-23 at most) and rounded to bf16: half a step is at most
2^-8 / (1 + 2^-8) < 2^-8 - 2^-17 of the value, so that 2^-8 holds both."""
import math

import pytest

import grouped_reference as gref

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, flush=True)


def make(sizes, types, seed, scale=1.0, shift=0):
    """Gradients as views that start `shift` elements into their storage."""
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = {"f": torch.float32, "b": torch.bfloat16}
    return [(torch.randn(n + shift, generator=g) * scale).to(dt[t]).cuda()[shift:] for n, t in zip(sizes, types)]


def workspace(grads):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    size = dense.etp_grad_norm_workspace(grads)
    return torch.full((size + 32,), 0xFF, dtype=torch.uint8, device="cuda"), size


def norm_of(grads):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    ws, size = workspace(grads)
    norm = torch.full((3,), -1.0, device="cuda")
    dense.etp_grad_norm(grads, norm[1:2], ws[:size] if size else None)
    torch.cuda.synchronize()
    assert (ws[size:] == 0xFF).all() and norm[0] == -1 and norm[2] == -1
    return float(norm[1])


def check_clipped(out, grads, scale):
    import torch
    for o, g in zip(out, grads):
        want = g.double() * scale
        step = 2.0 ** -24 + 2.0 ** -48 + (2.0 ** -8 if g.dtype == torch.bfloat16 else 0.0)
        assert o.dtype == g.dtype and ((o.double() - want).abs() <= want.abs() * step + 2.0 ** -149).all()


LISTS = [([1], "f"), ([1], "b"), ([3, 5, 7], "fbf"), ([0, 4, 0], "fbf"), ([8192], "f"), ([8193, 8191], "bf"),
         ([64 * 64, 64, 8 * 64, 64, 64, 64, 64 * 8, 8, 8 * 5 * 64], "f" * 9), ([100003, 17, 250001], "bfb"),
         ([1 + i % 50 for i in range(400)], "fb" * 200), ([300] * 120, "bf" * 60), ([32767, 1], "fb"), ([32768, 1], "fb"),
         ([511, 512, 513, 1024, 7], "fbfbb"), ([70000] * 121, "f" * 121), ([9000 + i for i in range(300)], "fbb" * 100),
         ([5_000_011, 12_345_678], "fb")]


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("sizes,types", LISTS)
def test_norm_and_clipping(sizes, types, shift):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("clip", len(sizes), sum(sizes), types[:3], shift)
    grads = make(sizes, types, sum(sizes), shift=shift)
    want = gref.grad_norm(grads)
    got = norm_of(grads)
    assert abs(got - want) <= want * (2.0 ** -24 + 2.0 ** -40)
    for most in (0.5 * want, 2.0 * want, 0.0):
        most = float(torch.tensor(most, dtype=torch.float32))
        scale = min(1.0, most / want)
        flat = [torch.full((g.numel() + 2,), 9.0, dtype=g.dtype, device="cuda") for g in grads]
        out = [t[1:-1] for t in flat]
        norm = torch.full((1,), -1.0, device="cuda")
        ws, size = workspace(grads)
        before = [g.clone() for g in grads]
        dense.etp_clip_grads(grads, most, out, norm, ws[:size] if size else None)
        torch.cuda.synchronize()
        assert float(norm) == got
        check_clipped(out, grads, scale)
        assert all((t[0] == 9).all() and (t[-1] == 9).all() for t in flat) and (ws[size:] == 0xFF).all()
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        # in place, through a list named once, and without the norm
        mine = dense.TensorList([g.clone() for g in grads])
        dense.etp_clip_grads(mine, most, None, None, ws[:size] if size else None)
        assert all(torch.equal(a, b) for a, b in zip(mine.tensors, out))


def test_no_tensors():
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("clip nothing")
    norm = torch.full((1,), -1.0, device="cuda")
    dense.etp_grad_norm([], norm)
    assert float(norm) == 0.0
    norm.fill_(-1.0)
    dense.etp_clip_grads([], 1.0, None, norm)
    assert float(norm) == 0.0
    dense.etp_clip_grads([], 1.0)
    empty = [torch.empty(0, device="cuda")]
    norm.fill_(-1.0)
    dense.etp_clip_grads(empty, 1.0, None, norm)
    assert float(norm) == 0.0


@pytest.mark.parametrize("size", [3e38, 1e30, 1e-30, 1e-44])
def test_squares_neither_overflow_nor_vanish(size):
    """Entries whose squares are no floats: the norm of n equal ones is sqrt(n) times one of them."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("clip range", size)
    n = 10007
    g = [torch.full((n,), size, device="cuda"), torch.full((5,), size, device="cuda").to(torch.bfloat16)]
    want = gref.grad_norm(g)
    if want < 3.4e38:
        assert abs(norm_of(g) - want) <= want * 2.0 ** -23 + 2.0 ** -149
    else:
        assert norm_of(g) == math.inf  # no float, but the scale is formed from the double
    out = [torch.empty_like(t) for t in g]
    dense.etp_clip_grads(g, 1.0, out, None, workspace(g)[0])
    check_clipped(out, g, min(1.0, 1.0 / want))


def test_non_finite_entries():
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("clip non-finite")
    for bad in (math.inf, -math.inf, math.nan):
        g = make([5000, 33, 9000], "fbf", 3)
        g[1][7] = bad
        out = [torch.empty_like(t) for t in g]
        norm = torch.zeros(1, device="cuda")
        dense.etp_clip_grads(g, 1.0, out, norm, workspace(g)[0])
        if math.isnan(bad):
            assert math.isnan(float(norm)) and all(torch.isnan(o).all() for o in out)
        else:
            assert float(norm) == math.inf and torch.isnan(out[1][7])
            out[1][7] = 0
            assert all((o == 0).all() for o in out)


def test_overlapping_outputs_are_refused():
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("clip overlap")
    flat = torch.ones(100, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        dense.etp_clip_grads([flat[:60], flat[50:]], 1.0, ws=ws)
    with pytest.raises(ValueError, match="overlap"):
        dense.etp_clip_grads([flat, flat], 1.0, ws=ws)
    assert abs(norm_of([flat, flat]) - 200 ** 0.5) < 1e-5  # the norm alone takes a tensor twice
    with pytest.raises(ValueError, match="types and sizes"):
        dense.etp_clip_grads([flat[:60]], 1.0, [flat[:61]], ws=ws)
    with pytest.raises(ValueError, match="types and sizes"):
        dense.etp_clip_grads([flat[:60]], 1.0, [flat[:60].bfloat16()], ws=ws)


def test_more_than_32_bits_of_entries():
    """One bf16 tensor of more than 2^31 entries: its end is read and scaled."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("clip 2^31")
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[0], g[n - 1], g[1 << 31] = 2.0, 4.0, 4.0
    ws = torch.empty(dense.etp_grad_norm_workspace([g]), dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")
    dense.etp_clip_grads([g], 3.0, None, norm, ws)
    assert float(norm) == 6.0
    assert float(g[0]) == 1.0 and float(g[n - 1]) == 2.0 and float(g[1 << 31]) == 2.0
    assert int((g != 0).sum()) == 3


def test_repeatable_on_a_stream_and_from_a_graph():
    """Bitwise equal calls, on another stream and replayed from a graph on new values, eager calls in between."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("clip graph")
    for sizes in ([500, 3, 77], [200000, 31, 70001, 5] * 50):
        grads = dense.TensorList(make(sizes, "fb" * len(sizes), 5))
        out = dense.TensorList([torch.empty_like(t) for t in grads.tensors])
        norm, ws = torch.empty(1, device="cuda"), workspace(grads)[0]
        dense.etp_clip_grads(grads, 1.0, out, norm, ws)
        first = [norm.clone(), *[t.clone() for t in out.tensors]]
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        dense.etp_clip_grads(grads, 1.0, out, norm, ws, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (norm, *out.tensors)))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dense.etp_clip_grads(grads, 1.0, out, norm, ws)
        for k in range(3):
            for t in grads.tensors:
                t.mul_(1.0 + 0.1 * k)
            dense.etp_clip_grads(grads, 1.0, out, norm, ws)
            want = [norm.clone(), *[t.clone() for t in out.tensors]]
            norm.fill_(-1)
            for t in out.tensors:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, (norm, *out.tensors))), k

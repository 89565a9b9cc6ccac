"""The dense operators together with the radial convolution as a user runs them
(examples/train_radial.py): gradients of the whole chain against differences,
and a training run that brings the loss down; and a captured HIP graph of the
same calls, replayed between eager work."""
import os
import sys

import pytest

import workloads

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def say(*a):
    print("[case]", *a, flush=True)


def test_training_lowers_the_loss():
    import train_radial
    say("train_radial tiny")
    losses = train_radial.train(steps=60)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.2 * losses[0] and min(losses) == min(losses[20:])


def test_chain_gradient_against_differences():
    """dLoss/dparameter along a random direction of each parameter, against central differences of the loss <G, out>
    (step 2^-6 and its half, extrapolated)."""
    import torch
    import train_radial as tr
    say("train_radial differences")
    layer = tr.Layer(workloads.get("tiny"))
    gen = torch.Generator(device="cuda").manual_seed(3)
    p = tr.parameters(layer.plan, gen)
    G = torch.randn(layer.out.shape, generator=gen, device="cuda")
    g = {k: torch.full_like(v, float("nan")) for k, v in p.items()}
    layer.forward(p)
    layer.backward(p, G, g)
    f = lambda q: float((layer.forward(q).double() * G.double()).sum())
    for k in p:
        d = torch.randn(p[k].shape, generator=gen, device="cuda")
        at = lambda t: f({**p, k: p[k] + t * d})
        h = 2.0 ** -6
        d1, d2 = (at(h) - at(-h)) / (2 * h), (at(h / 2) - at(-h / 2)) / h
        slope = float((g[k].double() * d.double()).sum())
        size = float(g[k].double().norm() * d.double().norm()) / d.numel() ** 0.5
        assert abs((4 * d2 - d1) / 3 - slope) < 2e-3 * max(size, abs(slope)), (k, d1, d2, slope, size)


def test_replays_of_a_captured_graph():
    """Forward, backward and update captured once (they allocate nothing and record no memset) and replayed; every
    replay equals the eager calls on the same parameters bit for bit."""
    import torch
    import train_radial as tr
    from equivariant_interatomic_potentials_amd import dense
    say("train_radial graph")
    layer = tr.Layer(workloads.get("tiny"))
    gen = torch.Generator(device="cuda").manual_seed(4)
    p = tr.parameters(layer.plan, gen)
    G = torch.randn(layer.out.shape, generator=gen, device="cuda")
    g = {k: torch.empty_like(v) for k, v in p.items()}
    X = torch.empty_like(p["W2"])
    ws = torch.empty(dense.etp_orthogonalize_workspace(1, *X.shape), dtype=torch.uint8, device="cuda")

    def calls():
        layer.forward(p)
        layer.backward(p, G, g)
        dense.etp_orthogonalize(g["W2"], X, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in range(4):
        for v in p.values():
            v.add_(torch.randn(v.shape, generator=gen, device="cuda"), alpha=0.05)
        calls()
        want = [layer.out.clone(), X.clone(), *[v.clone() for v in g.values()]]
        for t in (layer.out, X, *g.values()):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (layer.out, X, *g.values())):
            assert torch.equal(a, b), k

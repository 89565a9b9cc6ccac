"""Grouping, grouped layers, their gradients and clipping together with the radial
convolution as a user runs them (examples/train_elements.py): it runs, the chain's
gradients agree with differences, and a captured HIP graph of the calls replays
bit for bit between eager ones."""
import os
import sys

import numpy as np
import pytest

import grouped_reference as gref
import workloads

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def say(*a):
    print("[case]", *a, flush=True)


def setup(elements, seed):
    import torch
    import train_elements as te
    layer = te.Layer(workloads.get("tiny"), elements)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    p = te.parameters(layer.plan, elements, gen)
    return te, layer, gen, p, {k: torch.full_like(v, float("nan")) for k, v in p.items()}


@pytest.mark.parametrize("elements", [1, 3, 20])
def test_training_runs(elements):
    """Loss and gradient norm of every step are numbers, and no step is longer than the largest norm allows."""
    import torch
    import train_elements as te
    say("train_elements", elements)
    seen = te.train(steps=5, elements=elements)
    assert len(seen) == 5 and all(v == v and abs(v) < float("inf") for s in seen for v in s)
    te, layer, gen, p, g = setup(elements, 1)
    layer.backward(p, layer.forward(p).clone() * 100.0, g)
    opt = te.Optimiser(p, g)
    was = {k: v.clone() for k, v in p.items()}
    opt.step()
    assert float(opt.norm) > te.MAX_NORM
    assert abs(float(opt.norm) - gref.grad_norm(g.values())) <= float(opt.norm) * 2.0 ** -23
    moved = gref.grad_norm([was[k] - p[k] for k in p])
    assert moved <= opt.rate * te.MAX_NORM * (1 + 1e-5) + 1e-5  # (the difference of parameters of size 1 rounds at 2^-24)


def test_chain_gradient_against_differences():
    """dLoss/dparameter along a random direction of each parameter, against central differences of the loss <G, s>
    (step 2^-6 and its half, extrapolated)."""
    import torch
    say("train_elements differences")
    te, layer, gen, p, g = setup(3, 3)
    G = torch.randn(layer.s.shape, generator=gen, device="cuda")
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


def test_groups_are_the_elements():
    """The pairs' order is the stable sort of the edges by destination's and source's element."""
    wl = workloads.get("tiny")
    say("train_elements groups")
    te, layer, *_ = setup(3, 0)
    element = np.random.default_rng(0).integers(0, 3, wl.n)
    dst = np.repeat(np.arange(wl.n_dst), np.diff(wl.row_ptr))
    for (ptr, order), ids, n in ((layer.atoms, element[:wl.n_dst], 3), (layer.pairs, element[dst] * 3 + element[wl.src], 9)):
        want = gref.group_rows(ids, n)
        assert np.array_equal(ptr.cpu().numpy(), want[0]) and np.array_equal(order.cpu().numpy(), want[1])


def test_replays_of_a_captured_graph():
    """Forward, backward and clipping captured once and replayed on other parameters."""
    import torch
    say("train_elements graph")
    te, layer, gen, p, g = setup(4, 4)
    opt = te.Optimiser(p, g)
    G = torch.randn(layer.s.shape, generator=gen, device="cuda")

    def calls():
        layer.forward(p)
        layer.backward(p, G, g)
        te.dense.etp_clip_grads(opt.grads, 0.5, opt.into, opt.norm, opt.ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    outputs = (layer.s, opt.clipped, opt.norm, *g.values())
    for k in range(4):
        for v in p.values():
            v.add_(torch.randn(v.shape, generator=gen, device="cuda"), alpha=0.05)
        calls()
        want = [t.clone() for t in outputs]
        for t in outputs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outputs):
            assert torch.equal(a, b), k

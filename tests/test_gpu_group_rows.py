"""GPU parity of etp_group_rows with a stable sort on the host: every integer
equal, for one and two passes, one workgroup and many, padding, empty groups."""
import numpy as np
import pytest

import grouped_reference as gref

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, flush=True)


def group(ids, G, stream=None):
    import torch
    from equivariant_interatomic_potentials_amd import dense
    M = len(ids)
    t = torch.from_numpy(ids.astype(np.int32)).cuda()
    ptr = torch.full((G + 3,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((M + 2,), -7, dtype=torch.int32, device="cuda")
    size = dense.etp_group_rows_workspace(M, G)
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    dense.etp_group_rows(t, ptr[:G + 1], order[:M], ws[:size] if size else None, stream=stream)
    torch.cuda.synchronize()
    assert (ws[size:] == 0xFF).all() and (ptr[G + 1:] == -7).all() and (order[M:] == -7).all()
    return ptr[:G + 1].cpu().numpy(), order[:M].cpu().numpy()


def check(ids, G, **kw):
    ptr, order = group(ids, G, **kw)
    want_ptr, want_order = gref.group_rows(ids, G)
    assert np.array_equal(ptr, want_ptr)
    assert np.array_equal(order, want_order)


SIZES = [0, 1, 2, 63, 64, 65, 255, 1000, 4095, 4096, 4097, 5184, 16384, 16385, 20481, 100003, 441172]


@pytest.mark.parametrize("G", [1, 2, 5, 64, 100, 254, 255, 256, 257, 1000, 4000, 65535])
@pytest.mark.parametrize("M", SIZES)
def test_uneven_groups(M, G):
    say("group_rows", M, G)
    rng = np.random.default_rng(M + 7 * G)
    check((rng.random(M) ** 3 * G).astype(np.int64), G)


@pytest.mark.parametrize("G", [3, 255, 256, 700])
@pytest.mark.parametrize("M", [200, 5000, 30011])
def test_padding_and_empty_groups(M, G):
    """Ids outside 0 .. G - 1 (the lowest and the highest integer among them) come last; most groups are empty."""
    say("group_rows padding", M, G)
    rng = np.random.default_rng(M + G)
    ids = rng.choice([0, G - 1, G // 2, -1, G, 2 ** 31 - 1, -2 ** 31, G + 255, 65536], M)
    check(ids, G)
    check(np.full(M, -5), G)
    check(np.full(M, G - 1), G)


@pytest.mark.parametrize("G", [6, 7, 300, 65535])
@pytest.mark.parametrize("M", [3, 1023, 1024, 8191, 8192, 8193, 30011])
def test_long_runs_of_empty_groups(M, G):
    """Runs of empty groups in front, behind and between, shorter and longer than a lane or a wave writes at once."""
    say("group_rows empty runs", M, G)
    for at in ([0], [G - 1], [4, 5], [0, 4, G - 1], [0, 5, G - 1], [G // 2], [1, 65 % G, 131 % G, G // 3]):
        check(np.resize(np.array(at, dtype=np.int64), M), G)
        check(np.resize(np.array(at + [-1, G], dtype=np.int64), M), G)


@pytest.mark.parametrize("M,G", [(5172508, 100), (3000001, 1000)])
def test_many_rows(M, G):
    say("group_rows many", M, G)
    rng = np.random.default_rng(3)
    check(rng.integers(-2, G + 1, M), G)


def test_sorted_and_reversed_ids():
    say("group_rows sorted")
    ids = np.sort(np.random.default_rng(1).integers(0, 40, 50000))
    check(ids, 40)
    check(ids[::-1].copy(), 40)


def test_on_a_stream_and_from_a_graph():
    """Captured once and replayed on other ids, with eager calls in between."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("group_rows graph")
    s = torch.cuda.Stream()
    check(np.random.default_rng(2).integers(0, 30, 40000), 30, stream=s)
    for M, G in ((6000, 20), (50000, 20), (50000, 600)):
        ids = torch.zeros(M, dtype=torch.int32, device="cuda")
        ptr = torch.empty(G + 1, dtype=torch.int32, device="cuda")
        order = torch.empty(M, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(16, dense.etp_group_rows_workspace(M, G)), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dense.etp_group_rows(ids, ptr, order, ws)
        for k in range(3):
            new = np.random.default_rng(k).integers(-1, G, M)
            ids.copy_(torch.from_numpy(new.astype(np.int32)))
            ws.fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            want = gref.group_rows(new, G)
            assert np.array_equal(ptr.cpu().numpy(), want[0]) and np.array_equal(order.cpu().numpy(), want[1])
            check(new[::-1].copy(), G)

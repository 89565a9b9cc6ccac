"""etp_group_rows on more rows than its 2048 workgroups take in one tile of 4096 each, against a stable sort on the
device: a workgroup then places several tiles and carries its counts from one to the next."""
import pytest

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, flush=True)


@pytest.mark.parametrize("M,G", [(8388608, 100), (8388609, 100), (8388609, 1000), (20000003, 100), (20000003, 1000),
                                 (16777216, 255), (12345679, 65535)])
def test_several_tiles_a_workgroup(M, G):
    """Uneven groups and padding on both sides of the range, ends inside a tile."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    say("group_rows several tiles", M, G)
    g = torch.Generator(device="cuda").manual_seed(M + G)
    u = torch.rand(M, generator=g, device="cuda", dtype=torch.float64)
    ids = (u * u * (G + 3)).to(torch.int32) - 1  # -1, G and G + 1 among them
    ptr = torch.full((G + 3,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((M + 2,), -7, dtype=torch.int32, device="cuda")
    size = dense.etp_group_rows_workspace(M, G)
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        dense.etp_group_rows(ids, ptr[:G + 1], order[:M], ws[:size])
        key, want = torch.sort(torch.where((ids < 0) | (ids >= G), G, ids), stable=True)
        assert torch.equal(order[:M].long(), want)
        starts = torch.searchsorted(key, torch.arange(G + 1, dtype=torch.int32, device="cuda"))
        assert torch.equal(ptr[:G + 1].long(), starts)
        assert (ws[size:] == 0xFF).all() and (ptr[G + 1:] == -7).all() and (order[M:] == -7).all()
        ids = ids.flip(0).contiguous()

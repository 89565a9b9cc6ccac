"""Workspaces of the grouped layer's VJP: no partial sums where one run of rows holds every group."""
import pytest
import torch

from equivariant_interatomic_potentials_amd import dense


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,groups,n_in,n_out", [(2, 1, 65536, 16384), (1, 1, 64, 64), (31, 1, 128, 128),
                                                    (900, 40, 4096, 4096), (300, 3, 2048, 2048)])
def test_one_run_needs_no_partial_sums(rows, groups, n_in, n_out, dtype):
    """What is left is d (float), which layers of more than 128 inputs and outputs keep, and the bias gradient's parts
    where it is asked for alone: two for each run, of which there are at most rows / 32 + groups."""
    d = 4 * rows * n_out if n_in > 128 and n_out > 128 else 0
    bias = 2 * 4 * (rows // 32 + groups) * 2 * n_out
    assert dense.etp_grouped_linear_vjp_workspace(rows, groups, n_in, n_out, dtype) <= max(d, bias) + 16

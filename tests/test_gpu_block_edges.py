"""The dense block where rows are few, long, uneven or shared: sums that have one exact value, batches of which few rows are
in a group, workspaces of captured graphs, calls from several threads, outputs that would overlap inputs."""

import numpy as np
import pytest

import update_merged_table_gb300 as mt
import block_reference as R
from test_gpu_block import check_backward, norm_case, values, wide

pytestmark = pytest.mark.gpu


# ---- few rows in groups -----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("n,sizes,lead", [(5000, [3], 0), (5000, [1, 0, 2], 4990), (100_000, [40, 0, 1, 300], 7), (70_000, [0, 0], 5)])
@pytest.mark.parametrize("d,kind", [(64, "rms"), (1024, "layer")])
def test_norm_gradients_when_few_rows_are_in_groups(n, sizes, lead, d, kind):
    """The parameter gradients hold the groups' rows and nothing else, whatever the workspace held before."""
    rows, p, off = norm_case(31, sizes, lead, n - lead - sum(sizes), d, "bf16", "silu")
    nb = mt.GatedNorm(d, num_groups=len(sizes), kind=kind)
    nb.reserve_workspace(n)
    for t in nb._ws.values():
        t.fill_(255)  # NaN in fp32
    args = (rows["dz"], rows["dh"], rows["y"], rows["u"], rows["z"])
    got = nb.backward(*args, p, off)
    a, b = lead, lead + sum(sizes)
    inside = [wide(t[a:b]) for t in args]
    ref, size = R.norm_backward(*inside, values(p), wide(off).astype(np.int64) - a, kind, "silu", 1e-6)
    whole = mt.block.NormGrads(got.dx[a:b], got.dy[a:b], got.du[a:b], got.params)
    check_backward(nb, whole, ref, size, "bf16", max(sizes))
    for t in (got.dx, got.dy, got.du):
        assert not t[:a].any() and not t[b:].any()

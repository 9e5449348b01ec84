"""The dense block where rows are few, long, uneven or shared: sums that have one exact value, batches of which few rows are
in a group, workspaces of captured graphs, calls from several threads, outputs that would overlap inputs."""

import numpy as np
import pytest
import torch

import update_merged_table_gb300 as mt
import block_reference as R
from test_gpu_block import DEV, F, check_backward, near, norm_case, offsets_of, rand, values, wide

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


@pytest.mark.parametrize("n", [262_144 + 37])
def test_a_launch_of_many_milliseconds_reports_no_error(n):
    """Pairs of blocks at work for 20 ms and more: what a block waits for until the launch's end is no fault."""
    k = m = 8192
    gen = torch.Generator(device=DEV).manual_seed(41)
    x, w, dy = rand(gen, n, k), rand(gen, 2, m, k, scale=k ** -0.5), rand(gen, n, m)
    lin, off = mt.GroupedLinear(2, k, m), offsets_of([n - 101, 101])
    y = lin.forward(x, w, off)
    assert lin.error() == 0
    at = [0, 1, 131_000, n - 102, n - 101, n - 1]
    for g, rows in ((0, at[:4]), (1, at[4:])):
        want, size = wide(x[rows]) @ wide(w[g, :64]).T, np.abs(wide(x[rows])) @ np.abs(wide(w[g, :64])).T
        near(y[rows, :64], want, 2.0 ** -8 * np.abs(want) + (k + 16) * F * size)
    del y
    _, dw = lin.backward(dy, x, w, off, want_dx=False)
    assert lin.error() == 0
    for g, (a, b) in enumerate(((0, n - 101), (n - 101, n))):
        want = (dy[a:b, -8:].double().T @ x[a:b, -8:].double()).cpu().numpy()
        # sums of 512 rows are cut off at each step of 16 rows (2^-23 of the sum at most), and added up in fp32
        near(dw[g, -8:, -8:], want, (32 + n / 512) * F * np.sqrt(n) * 4, "dw")

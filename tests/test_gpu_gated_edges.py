"""The gated feed-forward part where a call's outputs or widths leave the common path; tolerances as in test_gpu_gated."""
import pytest
import torch

import update_merged_table_gb300 as mt
from test_gpu_gated import DEV, check_all, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,k,m", [([700, 0, 90], 64, 128), ([300, 5], 264, 40), ([2000] * 8, 512, 1024), ([1], 8, 8), ([9001, 300], 72, 512)])
def test_dx_on_any_element(sizes, k, m):
    """Rows of dx that start on one element, or lie an odd number of elements apart: the same products, so the same bits."""
    x, w, dh, off = make(21, sizes, 2, 3, "bf16", k, m)
    lin, h, (dx, dw) = check_all(x, w, dh, off, "bf16", "silu")
    n = x.shape[0]
    flat = torch.full((n * k + 2,), 7.0, device=DEV, dtype=torch.bfloat16)
    got = lin.backward(dh, x, w, off, want_dw=False, out_dx=flat[1:-1].view(n, k))[0]
    assert torch.equal(got, dx) and float(flat[0]) == 7 and float(flat[-1]) == 7
    big = torch.full((n, k + 9), 7.0, device=DEV, dtype=torch.bfloat16)
    for lo in (0, 3):
        got = lin.backward(dh, x, w, off, want_dw=False, out_dx=big[:, lo:lo + k])[0]
        assert torch.equal(got, dx) and (big[:, :lo] == 7).all() and (big[:, lo + k:] == 7).all()
        big.fill_(7.0)
    assert lin.error() == 0


@pytest.mark.parametrize("dtype,k,m", [("bf16", 72, 136), ("f32", 40, 48)])
def test_as_many_groups_as_there_may_be(dtype, k, m):
    """1024 groups, most of them of a few rows or of none, one long."""
    sizes = [(i * 7919) % 5 for i in range(1024)]
    sizes[77] = 700
    x, w, dh, off = make(22, sizes, 1, 2, dtype, k, m)
    check_all(x, w, dh, off, dtype, "gelu")


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Rows of every operand more than 2^31 elements apart from their first."""
    n, k, m, ld = 70000, 64, 96, 40000
    x, w, dh, off = make(23, [1000, n - 1003], 1, 2, "bf16", k, m)
    lin, h, (dx, dw) = check_all(x, w, dh, off, "bf16", "silu")
    big = torch.empty(n, ld, device=DEV, dtype=torch.bfloat16)
    part = [big[:, 1024 * i:1024 * i + c] for i, c in enumerate((k, m, m, k))]
    part[0].copy_(x), part[1].copy_(dh)
    assert torch.equal(lin.forward(part[0], w, off, out=part[2]), h)
    got = lin.backward(part[1], part[0], w, off, out_dx=part[3])
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    odd = big[:, 20001:20001 + k]  # rows on one element
    assert torch.equal(lin.backward(part[1], part[0], w, off, want_dw=False, out_dx=odd)[0], dx)

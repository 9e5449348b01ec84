"""A loss over the table's rows of a batch's own items, as the documents have it: IDs that come several times, and one that is
no ID."""
import pytest
import torch

import update_merged_table_gb300 as mt
from test_gpu_loss import DEV, check_all

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("row_dtype,dim,n,table_id", [("bf16", 64, 3000, 0), ("f32", 32, 500, 0), ("bf16", 16, 40, 7)])
def test_items_of_a_batch_are_the_vocabulary(row_dtype, dim, n, table_id):
    table = mt.Table(14, dim, row_dtype=row_dtype, init_scale=1.0, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    ids = (torch.rand(n, generator=gen, device=DEV).square() * (n // 3)).long()  # most come several times
    ids[5] = -7
    res = table.lookup(ids, [0, n], [table_id], gather=False)
    U = res.U
    assert 1 < U < n
    items = table.lookup(res.unique_keys[:U] & ((1 << 56) - 1), [0, U], [table_id])
    assert table.error() == mt.MT_EKEY
    assert items.U == U and torch.equal(items.unique_keys[:U], res.unique_keys[:U]) and torch.equal(items.unique_rows[:U], res.unique_rows[:U])
    # a target's row is its ID's
    live = res.inverse >= 0
    assert torch.equal(live, ids >= 0)
    assert torch.equal(items.unique_keys[:U][res.inverse.long()[live]] & ((1 << 56) - 1), ids[live])
    x = (torch.randn(n, dim, generator=gen, device=DEV)).to(items.rows.dtype)
    s = {"x": x, "w": items.rows, "targets": res.inverse, "dloss": torch.full((n,), 1.0 / n, device=DEV)}
    handle, r, (dx, dw) = check_all(s, row_dtype, smoothing=0.1)
    assert not r.loss[5] and not dx[5].any()
    before = items.rows.clone()
    gsum = table.backward_adam(items, dw, lr=1e-2, want_gsum=True)
    assert torch.equal(gsum[:U], dw.float())
    after = table.lookup(res.unique_keys[:U] & ((1 << 56) - 1), [0, U], [table_id]).rows
    assert bool((after != before).any(1).all()) and bool(torch.isfinite(after).all())

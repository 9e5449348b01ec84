"""A training step as it is put together: rows of a merged table through the gated part, a loss against the table's rows of the
candidates, a teacher's top logits over the same rows, and every gradient back to where it belongs."""
import numpy as np
import pytest
import torch

import loss_reference as R
import update_merged_table_gb300 as mt
from update_merged_table_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("row_dtype,dim", [("bf16", 64), ("f32", 32)])
def test_step_over_a_table(row_dtype, dim):
    """Each result against 64 bits on the inputs that the part was given, within a few roundings of its type."""
    dt = torch.bfloat16 if row_dtype == "bf16" else torch.float32
    tol = 6e-3 if row_dtype == "bf16" else 2e-5  # 2-norms: two roundings of 2^-9, or sums in fp32
    table = mt.Table(18, dim, row_dtype=row_dtype, device=DEV)
    b = W.jagged_batch(0, users=24, features=3)
    off = torch.from_numpy(np.ascontiguousarray(b.feat_offsets, np.int64)).to(DEV)
    res = table.lookup(torch.from_numpy(b.ids).to(DEV), b.feat_offsets, b.table_ids)
    # candidates: distinct IDs of the first feature, whose rows are the vocabulary
    cand = torch.from_numpy(np.unique(b.ids[b.feat_offsets[0]:b.feat_offsets[1]])).to(DEV)
    vres = table.lookup(cand)
    v, n = cand.numel(), b.n
    gen = torch.Generator(device=DEV).manual_seed(0)
    x0 = (torch.randn(n, dim, generator=gen, device=DEV)).to(dt)  # (fresh rows are tiny: a residual stream around them)
    x = (res.rows.float() * 8 + x0.float()).to(dt)
    vocab = (vres.rows.float() * 8).to(dt)
    w = (torch.randn(3, 2 * dim, dim, generator=gen, device=DEV) * dim ** -0.5).to(dt)
    gated = mt.GatedLinear(3, dim, dim, gate="silu", dtype=row_dtype)
    h = gated.forward(x, w, off)
    ref = R.gated(x.double(), w.double(), off, "silu")
    assert rel(h, ref["h"]) < tol
    # the first feature's positions predict the next position's ID; the others have no target
    targets = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    a, e = int(b.feat_offsets[0]), int(b.feat_offsets[1])
    ids = torch.from_numpy(b.ids).to(DEV)
    targets[a:e - 1] = torch.searchsorted(cand, ids[a + 1:e]).to(torch.int32)
    live = int((targets >= 0).sum())
    cross, distill = mt.CrossEntropy(v, dim, dtype=row_dtype), mt.Distillation(v, dim, 5, scale=0.5, dtype=row_dtype)
    r = cross.forward(h, vocab, targets)
    top = torch.randint(0, v, (n, 5), generator=gen, device=DEV)
    top[targets < 0] = -1
    teacher = torch.randn(n, 5, generator=gen, device=DEV)
    k = distill.forward(h, vocab, top, teacher)
    g = torch.full((n,), 1.0 / live, device=DEV)
    dh, dv = cross.backward(g, h, vocab, targets, r.lse)
    dh2, dv2 = distill.backward(0.5 * g, h, vocab, top, teacher, k.lse)
    H, V = h.double(), vocab.double()
    want = R.loss(H, V, targets=targets, dloss=g.double())
    want2 = R.loss(H, V, 0.5, ids=top, logits=teacher.double(), dloss=0.5 * g.double())
    assert rel(r.loss, want["loss"]) < 1e-5 and rel(k.loss, want2["loss"]) < 1e-5
    for got, ref in ((dh, want["dx"]), (dv, want["dw"]), (dh2, want2["dx"]), (dv2, want2["dw"])):
        assert rel(got, ref) < tol
    d = (dh.float() + dh2.float()).to(dt)
    dx, dw = gated.backward(d, x, w, off)
    ref = R.gated(x.double(), w.double(), off, "silu", d.double())
    assert rel(dx, ref["dx"]) < tol and rel(dw, ref["dw"]) < tol
    before = table.read_rows(vres.unique_rows[:vres.U])[0].clone()
    table.backward_adam(vres, (dv.float() + dv2.float()).to(dt).contiguous(), lr=1e-3)
    table.backward_adam(res, dx, lr=1e-3)
    after = table.read_rows(vres.unique_rows[:vres.U])[0]
    assert bool((after != before).any()) and bool(torch.isfinite(after).all())
    assert table.error() == 0 and not gated.error() and not cross.error() and not distill.error()

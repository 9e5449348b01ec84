"""Workspaces that a captured graph uses outlive their replacement by larger ones."""
import gc
import weakref

import numpy as np
import pytest
import torch

import update_merged_table_gb300 as mt

pytestmark = pytest.mark.gpu


def test_table_keeps_the_workspace_of_a_graph():
    tab = mt.Table(14, 16)
    ids = torch.from_numpy(np.random.default_rng(4).integers(0, 3000, size=2000).astype(np.int64)).cuda()
    tab.reserve_workspaces(2000)
    eager = tab.lookup(ids)
    res = tab.new_result(2000)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        tab.lookup(ids, result=res)
    used, unused = weakref.ref(tab._ws["lookup"]), weakref.ref(tab._ws["backward"])
    tab.reserve_workspaces(400_000)
    gc.collect()
    assert used() is not None and used() is not tab._ws["lookup"]
    assert unused() is None  # no graph holds it
    g.replay()
    torch.cuda.synchronize()
    U = eager.U
    assert res.U == U and torch.equal(res.unique_keys[:U], eager.unique_keys[:U]) and torch.equal(res.rows, eager.rows)
    assert tab.error() == 0


def test_merged_tables_keep_the_workspace_of_a_graph():
    tabs = mt.MergedTables([(16, "f32", 4000), (32, "f32", 4000)])
    ids = torch.from_numpy(np.random.default_rng(5).integers(0, 1000, size=1200).astype(np.int64)).cuda()
    tabs.lookup(ids, [0, 700, 1200])
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        held = tabs.lookup(ids, [0, 700, 1200], insert_missing=False)
    used = weakref.ref(tabs._ws["lookup"])
    more = torch.arange(50_000, device="cuda")
    eager = tabs.lookup(more, [0, 20_000, 50_000], insert_missing=False)
    gc.collect()
    assert used() is not None and used() is not tabs._ws["lookup"]
    del eager
    g.replay()
    torch.cuda.synchronize()
    eager = tabs.lookup(ids, [0, 700, 1200], insert_missing=False)
    for a, b in zip(held, eager):
        assert a.U == b.U and torch.equal(a.rows, b.rows)

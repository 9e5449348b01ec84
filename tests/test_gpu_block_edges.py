"""The dense block where rows are few, long, uneven or shared: sums that have one exact value, batches of which few rows are
in a group, workspaces of captured graphs, calls from several threads, outputs that would overlap inputs."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import update_merged_table_gb300 as mt
import block_reference as R
from test_gpu_block import DEV, F, check_backward, near, norm_case, offsets_of, rand, rounding, row_tol, values, wide

pytestmark = pytest.mark.gpu


def small_integers(gen, *shape, dtype=torch.bfloat16):
    """Whole numbers in [-2, 2]: their products and the sums of up to four million of them are exact in fp32."""
    return torch.randint(-2, 3, shape, generator=gen, device=DEV).to(dtype)


def time_of(f):
    times = []
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return min(times[1:])


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


def test_norm_gradients_of_a_group_without_rows_are_zero():
    """Also where that group's parameters are not finite."""
    rows, p, off = norm_case(44, [20, 0, 13], 0, 0, 64, "bf16", "silu")
    for t in (p.scale, p.post_weight, p.post_bias):
        t[1] = float("inf")
    nb = mt.GatedNorm(64, num_groups=3)
    got = nb.backward(rows["dz"], rows["dh"], rows["y"], rows["u"], rows["z"], p, off).params
    for t in (got.post_weight, got.post_bias, got.scale, got.pre_weight, got.pre_bias):
        assert torch.equal(t[1], torch.zeros_like(t[1])) and torch.isfinite(t).all()


@pytest.mark.parametrize("d", [4096, 5000, 8192])
def test_norm_wide_rows_in_fp32(d):
    """Teams of several warps, rows loaded when they are used."""
    rows, p, off = norm_case(45, [5, 0, 70], 1, 2, d, "f32", "sigmoid")
    nb = mt.GatedNorm(d, num_groups=3, kind="layer", gate="sigmoid", dtype="f32")
    r = nb.forward(rows["x"], rows["y"], rows["u"], p, off)
    z, h = R.norm_forward(wide(rows["x"]), wide(rows["y"]), wide(rows["u"]), values(p), wide(off), "layer", "sigmoid", 1e-6)
    near(r.z, z, 4 * row_tol(z, "f32"))
    near(r.h, h, 4 * row_tol(h, "f32"))
    for saved in ((rows["y"], rows["u"], rows["z"]), tuple(mt.pack8(rows[k]) for k in ("y", "u", "z"))):
        seen = [R.unpack(t.codes.cpu().numpy(), t.exps.cpu().numpy()) if isinstance(t, mt.Packed8) else wide(t) for t in saved]
        ref, size = R.norm_backward(wide(rows["dz"]), wide(rows["dh"]), *seen, values(p), wide(off), "layer", "sigmoid", 1e-6)
        check_backward(nb, nb.backward(rows["dz"], rows["dh"], *saved, p, off), ref, size, "f32", 70)


# ---- sums with one exact value ------------------------------------------------------------------------------------------

EXACT = [
    ("bf16", 512, 1024, [9001, 0, 3, 20000]),     # pairs of blocks, several chunks
    ("bf16", 512, 1024, [7001, 12345, 654]),      # dx by pairs
    ("bf16", 64, 64, [100_003]),                  # one narrow tile
    ("bf16", 264, 272, [10000, 63, 129]),
    ("bf16", 104, 200, [5001, 1, 4097]),          # 8-bit rows that are widened first
    ("bf16", 33, 250, [6000, 5001]),              # fp32 pipes
    ("f32", 32, 128, [8192, 1, 30011]),
    ("f32", 129, 257, [3000, 5000]),
    ("f32", 16, 16, [300_001, 5]),
]


@pytest.mark.parametrize("dtype,k,m,sizes", EXACT)
def test_linear_sums_are_exact_on_whole_numbers(dtype, k, m, sizes):
    """Every row is counted once: on small whole numbers every sum is exact in fp32, whatever its order."""
    gen = torch.Generator(device=DEV).manual_seed(k + m)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    n, lead = sum(sizes) + 12, 5
    x, dy, w = small_integers(gen, n, k, dtype=t), small_integers(gen, n, m, dtype=t), small_integers(gen, len(sizes), m, k, dtype=t)
    off = offsets_of(sizes, lead)
    lin = mt.GroupedLinear(len(sizes), k, m, dtype=dtype)
    lin.reserve_workspace(n)
    for b in lin._ws.values():
        b.fill_(255)
    y, dx = torch.zeros(n, m, device=DEV, dtype=torch.float64), torch.zeros(n, k, device=DEV, dtype=torch.float64)
    dw = torch.zeros(len(sizes), m, k, device=DEV, dtype=torch.float64)
    for g, (a, b) in enumerate(R.spans(off.tolist())):
        y[a:b], dx[a:b] = x[a:b].double() @ w[g].double().T, dy[a:b].double() @ w[g].double()
        dw[g] = dy[a:b].double().T @ x[a:b].double()
    assert torch.equal(lin.forward(x, w, off), y.float().to(t))
    for saved in (x, mt.pack8(x)):
        gx, gw = lin.backward(dy, saved, w, off)
        assert torch.equal(gx, dx.float().to(t))
        assert torch.equal(gw, dw.float())
    assert lin.error() == 0


@pytest.mark.parametrize("d,dtype,kind", [(64, "bf16", "layer"), (1024, "bf16", "rms"), (50, "f32", "layer"), (4096, "bf16", "rms")])
def test_norm_bias_sums_are_exact_on_whole_numbers(d, dtype, kind):
    """dpre_bias sums dh, dpost_bias (no gate, no scale, no next norm) sums dz: each row once."""
    sizes = [9000, 1, 0, 12345] if d < 4096 else [700, 0, 1300]
    rows, p, off = norm_case(32, sizes, 10, 20, d, dtype, "none")
    gen = torch.Generator(device=DEV).manual_seed(33)
    dv = small_integers(gen, rows["x"].shape[0], d, dtype=rows["x"].dtype)
    want = torch.stack([dv[a:b].double().sum(0) for a, b in R.spans(off.tolist())]).float()
    nb = mt.GatedNorm(d, num_groups=len(sizes), kind=kind, gate="none", dtype=dtype)
    one = mt.NormParams(pre_weight=p.pre_weight, pre_bias=p.pre_bias)
    assert torch.equal(nb.backward(None, dv, z=rows["z"], params=one, offsets=off).params.pre_bias, want)
    one = mt.NormParams(post_weight=p.post_weight, post_bias=p.post_bias)
    assert torch.equal(nb.backward(dv, None, y=rows["y"], params=one, offsets=off).params.post_bias, want)


# ---- graphs and threads ---------------------------------------------------------------------------------------------------

def test_captured_calls_have_a_workspace_of_their_own(monkeypatch):
    """A captured backward holds memory that lives as long as its graph: what the handle keeps for eager calls may grow
    meanwhile, and a graph may be replayed on another stream beside them."""
    gen = torch.Generator(device=DEV).manual_seed(34)
    sizes, k, m = [500, 300], 64, 128
    x, w, dy, off = rand(gen, 800, k), rand(gen, 2, m, k, scale=k ** -0.5), rand(gen, 800, m), offsets_of(sizes)
    rows, p, noff = norm_case(35, sizes, 0, 0, 128, "bf16", "silu")
    lin, nb = mt.GroupedLinear(2, k, m), mt.GatedNorm(128, num_groups=2)
    args = (rows["dz"], rows["dh"], rows["y"], rows["u"], rows["z"])

    def step():
        g = nb.backward(*args, p, noff)
        return [g.dx, g.params.scale, g.params.pre_weight, *lin.backward(dy, x, w, off)]

    s = torch.cuda.Stream()
    lin.reserve_workspace(800, stream=s)
    nb.reserve_workspace(800, stream=s)
    want = step()
    torch.cuda.synchronize()
    used = []
    native = mt.block._native

    class Seen:
        def __getattr__(self, name):
            f = getattr(native, name)
            return lambda *a: (used.append(a[-1]), f(*a))[1]

    monkeypatch.setattr(mt.block, "_native", Seen())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = step()
    kept = {t.data_ptr() for h in (lin, nb) for t in h._ws.values()}
    assert len(used) == 2 and not kept & {t.data_ptr() for t in used}
    monkeypatch.undo()
    used.clear()
    lin.reserve_workspace(200_000, stream=s)
    nb.reserve_workspace(200_000, stream=s)
    other = torch.cuda.CUDAGraph()  # a capture begins by emptying the allocator's cache
    with torch.cuda.graph(other, stream=s):
        step()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))
    # nothing needs to be reserved before a capture
    fresh, third = mt.GroupedLinear(2, k, m), torch.cuda.CUDAGraph()
    with torch.cuda.graph(third, stream=s):
        got = fresh.backward(dy, x, w, off)
    third.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[3]) and torch.equal(got[1], want[4])


def test_calls_from_several_threads_with_different_group_counts():
    """One kernel launched with much and with little shared memory by threads of their own (the C calls run without the
    interpreter's lock)."""
    lib = mt.load_library()
    gen = torch.Generator(device=DEV).manual_seed(36)
    n, d = 64, 128
    x = rand(gen, n, d)
    bad = []

    def worker(groups):
        s = torch.cuda.Stream()
        off = offsets_of([n] + [0] * (groups - 1))
        w = torch.ones(groups, d, device=DEV)
        h, y, weight = torch.empty_like(x), torch.empty_like(x), torch.zeros(groups, d, d, device=DEV, dtype=torch.bfloat16)
        torch.cuda.synchronize()

        class Rows(ctypes.Structure):
            _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("codes", ctypes.c_void_p), ("exps", ctypes.c_void_p)]

        class Norm(ctypes.Structure):
            _fields_ = [("n", ctypes.c_int64), ("dim", ctypes.c_int32), ("groups", ctypes.c_int32), ("dtype", ctypes.c_int32),
                        ("kind", ctypes.c_int32), ("gate", ctypes.c_int32), ("eps", ctypes.c_float), ("offsets", ctypes.c_void_p),
                        ("status", ctypes.c_void_p)] + [(k, ctypes.c_void_p) for k in ("pw", "pb", "sc", "qw", "qb")]

        c = Norm(n, d, groups, mt.MT_BF16, 0, 0, 1e-6, off.data_ptr(), None, None, None, None, w.data_ptr(), None)
        rx, rh, none = Rows(x.data_ptr(), d), Rows(h.data_ptr(), d), Rows()
        for _ in range(4000):
            rc = lib.mt_gated_norm_forward(ctypes.byref(c), ctypes.byref(rx), ctypes.byref(none), ctypes.byref(none),
                                           ctypes.byref(none), ctypes.byref(rh), s.cuda_stream)
            rc2 = lib.mt_group_linear_forward(x.data_ptr(), d, weight.data_ptr(), off.data_ptr(), groups, n, d, d, mt.MT_BF16,
                                              y.data_ptr(), d, None, s.cuda_stream) if groups < 32 else 0
            if rc or rc2:
                bad.append((groups, rc, rc2))
        s.synchronize()

    threads = [threading.Thread(target=worker, args=(g,)) for g in (1, 1024, 3, 700)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, (len(bad), bad[:5])


# ---- long sums ---------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,n,k,m", [("f32", 1_970_003, 16, 16), ("bf16", 1_970_003, 24, 20), ("bf16", 1_970_003, 64, 64)])
def test_weight_gradient_of_one_long_group(dtype, n, k, m):
    """A chain of r adds of unit normal products is off by about 2^-24 * sqrt(r / 2) of its sum at most (each add by half a
    unit in the last place of a partial sum that grows like the square root of the terms).  No chain has more than 1024
    rows; the partial sums of those (at most n / 1024) make another."""
    gen = torch.Generator(device=DEV).manual_seed(37)
    x, dy = rand(gen, n, k, dtype=dtype), rand(gen, n, m, dtype=dtype)
    off = offsets_of([n])
    _, dw = mt.GroupedLinear(1, k, m, dtype=dtype).backward(dy, x, None, off, want_dx=False)
    want = sum(dy[a:a + 65536].double().T @ x[a:a + 65536].double() for a in range(0, n, 65536))
    off_by = (dw[0].double() - want).square().mean().sqrt() / want.square().mean().sqrt()
    assert off_by <= 2.0 ** -24 * np.sqrt((1024 + n / 1024) / 2), float(off_by)


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


@pytest.mark.parametrize("dtype,k,m", [("bf16", 64, 64), ("f32", 16, 16)])
def test_weight_gradient_of_one_long_group_takes_every_block(dtype, k, m):
    """One group, or one beside a small one, in no more than twice the time of 61 equal ones."""
    gen = torch.Generator(device=DEV).manual_seed(42)
    n = 61 * 16000
    x, dy = rand(gen, n, k, dtype=dtype), rand(gen, n, m, dtype=dtype)
    times = []
    for sizes in ([16000] * 61, [n], [100, n - 100]):
        lin, off = mt.GroupedLinear(len(sizes), k, m, dtype=dtype), offsets_of(sizes)
        times.append(time_of(lambda: lin.backward(dy, x, None, off, want_dx=False)))
    assert max(times[1:]) <= 2 * times[0], times


# ---- one group has all the rows of a batch that is small for its groups ---------------------------------------------------------

@pytest.mark.parametrize("dtype,groups,n,k,m", [("bf16", 256, 512, 512, 256), ("bf16", 64, 128, 512, 64), ("f32", 64, 512, 256, 128)])
def test_forward_of_few_rows_does_not_depend_on_their_group(dtype, groups, n, k, m):
    """All rows in one group: the same values, in no more than a few times the time of rows spread over the groups."""
    gen = torch.Generator(device=DEV).manual_seed(38)
    x, w = rand(gen, n, k, dtype=dtype), rand(gen, groups, m, k, dtype=dtype, scale=k ** -0.5)
    lin = mt.GroupedLinear(groups, k, m, dtype=dtype)
    even = offsets_of([n // groups] * groups)
    one = offsets_of([0] * 3 + [n] + [0] * (groups - 4))
    for off in (even, one):
        want, size = R.linear_forward(wide(x), wide(w), wide(off))
        near(lin.forward(x, w, off), want, rounding(dtype) * np.abs(want) + (k + 16) * F * size)
    out = torch.empty(n, m, device=DEV, dtype=x.dtype)
    spread, alone = (time_of(lambda o=o: lin.forward(x, w, o, out=out)) for o in (even, one))
    assert alone <= 4 * spread, (alone, spread)


def test_norm_gradients_of_many_groups_without_rows():
    """One row and 1024 groups: as much as the groups' gradients take to write, not a launch of blocks for each."""
    d = 2048
    times = []
    for groups in (8, 1024):
        rows, p, off = norm_case(43, [1] + [0] * (groups - 1), 0, 0, d, "bf16", "silu")
        nb = mt.GatedNorm(d, num_groups=groups)
        args = (rows["dz"], rows["dh"], rows["y"], rows["u"], rows["z"])
        got = nb.backward(*args, p, off).params
        assert got.post_weight[0].any() and not any(t[1:].any() for t in (got.post_weight, got.post_bias, got.scale, got.pre_weight, got.pre_bias))
        times.append(time_of(lambda: nb.backward(*args, p, off)))
    assert times[1] <= 24 * times[0], times


# ---- what a call refuses, and what it takes ---------------------------------------------------------------------------------------

def refused(f, *a, **kw):
    with pytest.raises(mt.MTError) as e:
        f(*a, **kw)
    assert e.value.code == mt.MT_EINVAL


def test_outputs_that_overlap_are_refused():
    t = dict(device=DEV, dtype=torch.bfloat16)
    n, d = 40, 64
    big = torch.zeros(n, 3 * d, **t)
    x, y, off = torch.zeros(n, d, **t), torch.zeros(n, d, **t), offsets_of([15, 25])
    w = torch.zeros(2, d, d, **t)
    lin = mt.GroupedLinear(2, d, d)
    refused(lin.forward, x, w, off, out=x)
    refused(lin.forward, big[:, :d], w, off, out=big[:, d - 1:2 * d - 1])
    refused(lin.forward, big[:-1, :d], w, offsets_of([15, 24]), out=big[1:, :d])
    refused(lin.forward, x, w, off, out=w.view(-1, d)[:n])
    refused(lin.backward, x, y, w, off, out_dx=x)
    refused(lin.backward, x, y, w, off, out_dx=w.view(-1, d)[:n])
    dw = torch.zeros(2, d, d, device=DEV)
    refused(lin.backward, x, dw.view(-1).view(torch.bfloat16)[:n * d].view(n, d), w, off, out_dw=dw)
    lin.forward(big[:, :d], w, off, out=big[:, d:2 * d])         # column slices of one tensor do not overlap
    lin.backward(big[:, :d], big[:, 2 * d:], w, off, out_dx=big[:, d:2 * d])
    lin.forward(big[0:20, :d], w, offsets_of([5, 15]), out=big[20:, :d])
    both = torch.zeros(2 * n, d, **t)
    lin.forward(both[0::2], w, off, out=both[1::2])              # nor do alternate rows
    one = mt.NormParams(post_weight=torch.ones(d, device=DEV), pre_weight=torch.ones(d, device=DEV))
    nb = mt.GatedNorm(d)
    refused(nb.forward, x, y, y, one, out_h=y)
    refused(nb.forward, x, y, y, one, out_z=big[:, :d], out_h=big[:, 8:8 + d])
    refused(nb.backward, x, x, y, y, y, one, out_dx=big[:, :d], out_dy=big[:, d // 2:d // 2 + d])
    refused(nb.backward, x, x, y, y, y, one, out_du=y)
    nb.backward(x, x, y, y, y, one, out_dy=big[:, :d], out_du=big[:, d:2 * d])
    p = mt.pack8(x)
    refused(mt.pack8, x, out=mt.Packed8(x.view(torch.int8).view(-1, d)[:n], p.exps))
    refused(mt.unpack8, mt.Packed8(x.view(torch.int8).view(-1, d)[:n], p.exps), out=x)


def test_one_row_of_any_stride():
    """A batch of one row: the distance to a next row that is not there does not matter."""
    gen = torch.Generator(device=DEV).manual_seed(39)
    x, w, off = rand(gen, 1, 64), rand(gen, 1, 32, 64), offsets_of([1])
    far = x.as_strided((1, 64), (1 << 31, 1))
    lin = mt.GroupedLinear(1, 64, 32)
    assert torch.equal(lin.forward(far, w, off), lin.forward(x, w, off))
    assert torch.equal(mt.pack8(far).codes, mt.pack8(x).codes)


def test_out_of_memory_is_the_error_of_torch():
    """Outputs that do not fit raise what torch raises, so that a caller can catch it."""
    x, w, off = torch.zeros(20_000_000, 1, device=DEV), torch.zeros(1, 8192, 1, device=DEV), offsets_of([20_000_000])
    with pytest.raises(torch.OutOfMemoryError):
        mt.GroupedLinear(1, 1, 8192, dtype="f32").forward(x, w, off)


def test_checkpoint_parts_that_do_not_belong_together_are_refused():
    gen = torch.Generator(device=DEV).manual_seed(40)
    p, q = mt.pack8(rand(gen, 50, 64)), mt.pack8(rand(gen, 5, 64))
    p.exps = q.exps
    with pytest.raises(ValueError):
        mt.unpack8(p)
    p.codes = p.codes[0]
    with pytest.raises(ValueError):
        mt.unpack8(p)

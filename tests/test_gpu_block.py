"""The dense block's operators (grouped products, gated norms, 8-bit checkpoints) against their 64-bit definitions.

Tolerances, fixed from the arithmetic:
* a bf16 result is rounded once from an fp32 value: at most 2^-8 of its size apart (half of that is the rounding; the
  rest covers a value next to a rounding boundary), plus the fp32 value's own error;
* a sum of k products in fp32 is at most k * 2^-23 of the sum of their absolute values off (a tensor core may truncate
  where an fp32 add rounds, hence 2^-23 and not 2^-24);
* a norm's value goes through at most 16 + 9 adds in a row per statistic and fewer than 40 further roundings: 64 * 2^-23
  of the row's size (its largest value stands for the size of what was added).
"""
import numpy as np
import pytest
import torch

import update_merged_table_gb300 as mt
import block_reference as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
F = 2.0 ** -23


def rounding(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23


def wide(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, want, tol, what=""):
    got = wide(got)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4],
                           np.broadcast_to(tol, want.shape)[bad][:4])


def rand(gen, *shape, dtype="bf16", scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(TORCH[dtype])


def offsets_of(sizes, lead=0):
    return torch.tensor(np.concatenate([[lead], lead + np.cumsum(sizes)]), dtype=torch.int64, device=DEV)


# ---- 8-bit checkpoints -----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 31), (5, 32), (7, 33), (4, 64), (129, 200), (33, 777), (2, 8192), (0, 64)])
def test_pack_matches_the_definition(dtype, n, d):
    gen = torch.Generator(device=DEV).manual_seed(n * 8192 + d)
    x = rand(gen, n, d, dtype=dtype) * torch.exp(8 * torch.randn(n, 1, generator=gen, device=DEV)).to(TORCH[dtype])
    p = mt.pack8(x)
    codes, exps = R.pack(wide(x))
    assert np.array_equal(p.codes.cpu().numpy(), codes)
    assert np.array_equal(p.exps.cpu().numpy(), exps)
    for out in ("bf16", "f32"):
        assert np.array_equal(wide(mt.unpack8(p, TORCH[out])), R.unpack(codes, exps))  # exact in both


def test_pack_edges():
    """Zeros, the largest and smallest numbers, exact ties, the boundary of the exponent, infinities and NaN."""
    big = float(torch.finfo(torch.float32).max)
    rows = torch.zeros(10, 70, device=DEV)
    rows[1] = big
    rows[2] = torch.finfo(torch.float32).tiny
    rows[3, :] = 1e-44                      # subnormal
    rows[4, 0], rows[4, 1:5] = 127.0, torch.tensor([0.5, 1.5, 2.5, -0.5], device=DEV)  # ties to even
    rows[5, 0] = 127.0 * 2.0 ** -3
    rows[6, 0] = float(np.nextafter(np.float32(127.0 * 2.0 ** -3), np.float32(np.inf)))
    rows[7, 3], rows[7, 40] = float("inf"), 1.0
    rows[8, 69], rows[8, 0] = float("nan"), -2.0
    rows[9] = -big
    p = mt.pack8(rows)
    codes, exps = R.pack(wide(rows))
    assert np.array_equal(p.codes.cpu().numpy(), codes)
    assert np.array_equal(p.exps.cpu().numpy(), exps)
    back = wide(mt.unpack8(p, torch.float32))
    assert np.array_equal(back, R.unpack(codes, exps), equal_nan=True)
    assert np.isnan(back[7, :32]).all() and np.isfinite(back[7, 32:]).all() and np.isnan(back[8, 64:]).all()
    assert np.isfinite(back[[1, 9]]).all()
    err = np.abs(back[:7] - wide(rows)[:7])
    step = np.ldexp(1.0, exps[:7].astype(int) - 127).repeat(32, 1)[:, :70]
    assert (err[2:] <= 0.5 * step[2:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pack_strided_and_unaligned_rows(dtype):
    gen = torch.Generator(device=DEV).manual_seed(3)
    big = rand(gen, 50, 160, dtype=dtype)
    for lo, hi in [(0, 64), (64, 160), (1, 65), (3, 100)]:
        x = big[:, lo:hi]
        p = mt.pack8(x)
        codes, exps = R.pack(wide(x))
        assert np.array_equal(p.codes.cpu().numpy(), codes) and np.array_equal(p.exps.cpu().numpy(), exps)
        out = torch.zeros_like(big)
        mt.unpack8(p, out=out[:, lo:hi])
        assert np.array_equal(wide(out[:, lo:hi]), R.unpack(codes, exps))
        assert not out[:, :lo].any() and not out[:, hi:].any()


# ---- grouped products ------------------------------------------------------------------------------------------------

SIZES = [
    ([1], 0, 0),
    ([0, 5, 0, 130, 1], 0, 0),
    ([0, 0], 3, 2),             # no row in any group
    ([64, 64], 0, 0),
    ([257, 0, 129, 300], 2, 3),  # rows before and after the groups
    ([3] * 61, 0, 0),
]
SHAPES = [("bf16", 64, 256), ("bf16", 8, 8), ("bf16", 72, 136), ("bf16", 50, 33), ("bf16", 512, 128), ("bf16", 1, 1),
          ("f32", 16, 64), ("f32", 50, 33), ("f32", 128, 200)]


def linear_case(seed, sizes, lead, tail, dtype, k, m):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = lead + sum(sizes) + tail
    return (rand(gen, n, k, dtype=dtype), rand(gen, len(sizes), m, k, dtype=dtype, scale=k ** -0.5),
            rand(gen, n, m, dtype=dtype), offsets_of(sizes, lead))


@pytest.mark.parametrize("sizes,lead,tail", SIZES)
@pytest.mark.parametrize("dtype,k,m", SHAPES)
def test_linear_forward_and_gradients(sizes, lead, tail, dtype, k, m):
    x, w, dy, off = linear_case(1, sizes, lead, tail, dtype, k, m)
    lin = mt.GroupedLinear(len(sizes), k, m, dtype=dtype)
    y = lin.forward(x, w, off)
    want, size = R.linear_forward(wide(x), wide(w), wide(off))
    near(y, want, rounding(dtype) * np.abs(want) + (k + 16) * F * size, "y")
    dx, dw = lin.backward(dy, x, w, off)
    wdx, sdx, wdw, sdw = R.linear_backward(wide(dy), wide(x), wide(w), wide(off))
    near(dx, wdx, rounding(dtype) * np.abs(wdx) + (m + 16) * F * sdx, "dx")
    near(dw, wdw, (max(sizes) + 16) * F * sdw, "dw")
    # from 8 bits: the product of the values that the checkpoint stands for
    p = mt.pack8(x)
    dx8, dw8 = lin.backward(dy, p, w, off)
    _, _, wdw, sdw = R.linear_backward(wide(dy), R.unpack(p.codes.cpu().numpy(), p.exps.cpu().numpy()), wide(w), wide(off))
    near(dw8, wdw, (max(sizes) + 16) * F * sdw, "dw from 8 bits")
    assert torch.equal(dx8, dx)
    assert lin.error() == 0
    # the same call gives the same bits
    again = lin.backward(dy, x, w, off)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(lin.forward(x, w, off), y)


@pytest.mark.parametrize("dtype,k,m,sizes", [
    ("bf16", 64, 256, [9001, 0, 3, 20000]), ("bf16", 256, 512, [5000, 4097, 4096]), ("bf16", 1024, 2048, [300, 700, 40]),
    ("bf16", 2048, 1024, [129, 2]), ("bf16", 264, 40, [10000]), ("f32", 32, 128, [8192, 1, 8192]),
    ("f32", 129, 257, [3000, 5000]), ("bf16", 33, 250, [6000, 5001])])
def test_linear_long_groups(dtype, k, m, sizes):
    """Groups split over several chunks, several tiles in every direction."""
    x, w, dy, off = linear_case(2, sizes, 5, 7, dtype, k, m)
    lin = mt.GroupedLinear(len(sizes), k, m, dtype=dtype)
    want, size = R.linear_forward(wide(x), wide(w), wide(off))
    near(lin.forward(x, w, off), want, rounding(dtype) * np.abs(want) + (k + 16) * F * size, "y")
    p = mt.pack8(x)
    for xx, xv in ((x, wide(x)), (p, R.unpack(p.codes.cpu().numpy(), p.exps.cpu().numpy()))):
        dx, dw = lin.backward(dy, xx, w, off)
        wdx, sdx, wdw, sdw = R.linear_backward(wide(dy), xv, wide(w), wide(off))
        near(dx, wdx, rounding(dtype) * np.abs(wdx) + (m + 16) * F * sdx, "dx")
        near(dw, wdw, (max(sizes) + 16) * F * sdw, "dw")


@pytest.mark.parametrize("k,m", [(256, 512), (512, 1024), (264, 272)])
def test_linear_many_short_groups(k, m):
    """More tiles than the SMs hold at once, most of them shorter than a stage of 64 rows: the short last stages of
    several chunks are on their way together."""
    sizes = [5, 70, 3, 64, 1, 130, 0, 63] * 12 + [700, 2000]
    x, w, dy, off = linear_case(4, sizes, 2, 1, "bf16", k, m)
    lin = mt.GroupedLinear(len(sizes), k, m)
    p = mt.pack8(x)
    for xx, xv in ((x, wide(x)), (p, R.unpack(p.codes.cpu().numpy(), p.exps.cpu().numpy()))):
        dx, dw = lin.backward(dy, xx, w, off)
        wdx, sdx, wdw, sdw = R.linear_backward(wide(dy), xv, wide(w), wide(off))
        near(dx, wdx, 2.0 ** -8 * np.abs(wdx) + (m + 16) * F * sdx, "dx")
        near(dw, wdw, (max(sizes) + 16) * F * sdw, "dw")
    assert lin.error() == 0


def test_linear_strided_rows_and_outputs():
    """Column slices of wider tensors as inputs and outputs, aligned and not; what lies beside them stays."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    for lo in (0, 8, 3):
        k, m, sizes = 64, 96, [100, 60]
        big_x, big_dy = rand(gen, 160, 200), rand(gen, 160, 300)
        x, dy = big_x[:, lo:lo + k], big_dy[:, lo:lo + m]
        w, off = rand(gen, 2, m, k, scale=k ** -0.5), offsets_of(sizes)
        lin = mt.GroupedLinear(2, k, m)
        big_y, big_dx = torch.full((160, 128), 7.0, device=DEV, dtype=torch.bfloat16), torch.full((160, 80), 7.0, device=DEV, dtype=torch.bfloat16)
        lin.forward(x, w, off, out=big_y[:, lo:lo + m])
        dx, dw = lin.backward(dy, x, w, off, out_dx=big_dx[:, lo:lo + k])
        want, size = R.linear_forward(wide(x), wide(w), wide(off))
        near(big_y[:, lo:lo + m], want, 2.0 ** -8 * np.abs(want) + (k + 16) * F * size)
        wdx, sdx, wdw, sdw = R.linear_backward(wide(dy), wide(x), wide(w), wide(off))
        near(dx, wdx, 2.0 ** -8 * np.abs(wdx) + (m + 16) * F * sdx)
        near(dw, wdw, 116 * F * sdw)
        assert (big_y[:, :lo] == 7).all() and (big_y[:, lo + m:] == 7).all()
        assert (big_dx[:, :lo] == 7).all() and (big_dx[:, lo + k:] == 7).all()


def test_linear_not_a_number_stays_in_its_row_and_group():
    """A NaN or infinity in one row reaches that row of y and its group's dW only: not the next group's tile mates."""
    sizes, k, m = [70, 50, 40], 64, 64
    x, w, dy, off = linear_case(6, sizes, 3, 4, "bf16", k, m)
    x[3 + 69, 5], dy[3 + 70, 7] = float("nan"), float("inf")  # the last row of group 0, the first of group 1
    x[1], x[-2] = float("nan"), float("inf")                  # rows in no group
    lin = mt.GroupedLinear(3, k, m)
    y = lin.forward(x, w, off)
    dx, dw = lin.backward(dy, x, w, off)
    assert torch.isnan(y[72]).all() and torch.isfinite(y[:72]).all() and torch.isfinite(y[73:]).all()
    assert not torch.isfinite(dx[73]).any() and torch.isfinite(dx[:73]).all() and torch.isfinite(dx[74:]).all()
    assert torch.isnan(dw[0, :, 5]).all() and torch.isfinite(dw[0, :, :5]).all() and torch.isfinite(dw[0, :, 6:]).all()
    assert not torch.isfinite(dw[1, 7]).any() and torch.isfinite(dw[1, :7]).all() and torch.isfinite(dw[1, 8:]).all()
    assert torch.isfinite(dw[2]).all()
    _, dw8 = lin.backward(dy, mt.pack8(x), w, off)
    assert torch.isnan(dw8[0, :, :32]).all() and torch.isfinite(dw8[0, :, 32:]).all() and torch.isfinite(dw8[2]).all()


@pytest.mark.parametrize("bad", [[0, 40, 20, 100], [-5, 10, 50, 100], [0, 10, 50, 4000], [100, 0, 0, 0],
                                 [2 ** 62, -2 ** 62, 2 ** 40, 50]])
@pytest.mark.parametrize("k", [64, 33])
def test_linear_bad_offsets_latch(bad, k):
    gen = torch.Generator(device=DEV).manual_seed(7)
    x, w, dy = rand(gen, 100, k), rand(gen, 3, 64, k), rand(gen, 100, 64)
    off = torch.tensor(bad, dtype=torch.int64, device=DEV)
    lin = mt.GroupedLinear(3, k, 64)
    y = lin.forward(x, w, off)
    dx, dw = lin.backward(dy, x, w, off)
    ref = R.safe_offsets(bad, 100)
    want, size = R.linear_forward(wide(x), wide(w), ref)
    near(y, want, 2.0 ** -8 * np.abs(want) + (k + 16) * F * size)
    _, _, wdw, sdw = R.linear_backward(wide(dy), wide(x), wide(w), ref)
    near(dw, wdw, 116 * F * sdw)
    assert lin.error(clear=True) == mt.MT_EINVAL and lin.error() == 0


def test_linear_empty_batch_and_parts():
    w = torch.ones(3, 16, 8, device=DEV, dtype=torch.bfloat16)
    off = torch.zeros(4, dtype=torch.int64, device=DEV)
    lin = mt.GroupedLinear(3, 8, 16)
    x, dy = torch.empty(0, 8, device=DEV, dtype=torch.bfloat16), torch.empty(0, 16, device=DEV, dtype=torch.bfloat16)
    assert lin.forward(x, w, off).shape == (0, 16)
    dx, dw = lin.backward(dy, x, w, off)
    assert dx.shape == (0, 8) and dw.shape == (3, 16, 8) and not dw.any()
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, dy, off = rand(gen, 20, 8), rand(gen, 20, 16), offsets_of([5, 5, 10])
    dx, dw = lin.backward(dy, x, w, off)
    only_dx, none = lin.backward(dy, None, w, off, want_dw=False)
    assert none is None and torch.equal(only_dx, dx)
    none, only_dw = lin.backward(dy, x, None, off, want_dx=False)
    assert none is None and torch.equal(only_dw, dw)


def test_linear_gradients_against_differences():
    """<dW, V> and <dx, V> against central differences of <c, y> in 64 bits (y is linear in each: only rounding is left)."""
    x, w, c, off = linear_case(8, [30, 0, 50], 0, 0, "f32", 24, 40)
    lin = mt.GroupedLinear(3, 24, 40, dtype="f32")
    dx, dw = lin.backward(c, x, w, off)
    rng = np.random.default_rng(0)
    X, W, C, O = wide(x), wide(w), wide(c), wide(off)
    for grad, which in ((dx, 0), (dw, 1)):
        V = rng.standard_normal(grad.shape)
        step = 1e-3

        def loss(sign):
            d = sign * step * V
            y = R.linear_forward(X + d, W, O)[0] if which == 0 else R.linear_forward(X, W + d, O)[0]
            return (C * y).sum()

        diff = (loss(1) - loss(-1)) / (2 * step)
        got = (wide(grad) * V).sum()
        assert abs(got - diff) <= 1e-6 * (np.abs(wide(grad)) * np.abs(V)).sum()


# ---- gated norm -------------------------------------------------------------------------------------------------------

def norm_case(seed, sizes, lead, tail, d, dtype, gate, bias=True, scale=True):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n, g = lead + sum(sizes) + tail, len(sizes)
    rows = {k: rand(gen, n, d, dtype=dtype, scale=s) for k, s in (("x", 1.0), ("y", 2.0), ("u", 1.5), ("z", 1.5), ("dz", 1.0), ("dh", 1.0))}
    if gate == "none":
        rows["u"] = None

    def param(mean, spread):
        return mean + spread * torch.randn(g, d, generator=gen, device=DEV)

    p = mt.NormParams(param(1.0, 0.3), param(0.0, 0.3) if bias else None, param(0.5, 0.2) if scale else None,
                      param(1.0, 0.3), param(0.0, 0.3) if bias else None)
    return rows, p, offsets_of(sizes, lead)


def values(p):
    return {k: wide(getattr(p, k)) for k in ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")}


def row_tol(want, dtype):
    """Per row: the rounding of the result, and 64 roundings in fp32 of values of the row's size."""
    top = np.abs(want).max(1, keepdims=True) if want.size else 0.0
    return rounding(dtype) * np.abs(want) + 64 * F * (top + 1.0)


def check_backward(nb, got, ref, size, dtype, rows):
    want = {"dx": got.dx, "dy": got.dy, "du": got.du}
    for k, t in want.items():
        assert (t is None) == (k not in ref)
        if t is not None:
            near(t, ref[k], 4 * row_tol(ref[k], "f32") + rounding(dtype) * np.abs(ref[k]), k)
    for k in ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias"):
        t = getattr(got.params, k)
        assert (t is None) == (k not in ref)
        if t is not None:
            # each term is a few roundings off (64 * F), and so is the sum over a team's rows
            near(t, ref[k], (64 + rows / 16) * F * (size[k] + 1e-6), k)


NORM_SIZES = [([1], 0, 0), ([0, 3, 0, 17, 1], 0, 0), ([0, 0], 2, 1), ([400, 0, 129], 3, 2), ([2] * 61, 0, 0)]


@pytest.mark.parametrize("sizes,lead,tail", NORM_SIZES)
@pytest.mark.parametrize("d,dtype,kind,gate,bias,scale", [
    (512, "bf16", "rms", "silu", False, True), (64, "bf16", "layer", "sigmoid", True, True), (16, "f32", "layer", "silu", True, False),
    (1, "f32", "rms", "linear", False, False), (50, "bf16", "layer", "none", True, True), (777, "f32", "rms", "sigmoid", True, True),
    (1024, "bf16", "layer", "linear", True, False), (33, "bf16", "rms", "silu", False, True), (2048, "f32", "rms", "silu", False, True)])
def test_norm_forward_and_gradients(sizes, lead, tail, d, dtype, kind, gate, bias, scale):
    rows, p, off = norm_case(11, sizes, lead, tail, d, dtype, gate, bias, scale)
    nb = mt.GatedNorm(d, num_groups=len(sizes), kind=kind, gate=gate, eps=1e-5, dtype=dtype)
    r = nb.forward(rows["x"], rows["y"], rows["u"], p, off, pack="yuzh" if gate != "none" else "yzh")
    v, o = values(p), wide(off)
    z, h = R.norm_forward(wide(rows["x"]), wide(rows["y"]), wide(rows["u"]), v, o, kind, gate, 1e-5)
    near(r.z, z, 4 * row_tol(z, "f32") + rounding(dtype) * np.abs(z), "z")
    near(r.h, h, 4 * row_tol(h, "f32") + rounding(dtype) * np.abs(h), "h")
    inside = torch.zeros(rows["x"].shape[0], 1, dtype=torch.bool, device=DEV)
    inside[int(o[0]):int(o[-1])] = True
    for k, t in (("y", rows["y"]), ("u", rows["u"]), ("z", r.z), ("h", r.h)):
        if k in r.packed:  # the bytes that pack8 makes of the rows (zeros for rows in no group)
            q = mt.pack8(torch.where(inside, t, torch.zeros_like(t)))
            assert torch.equal(q.codes, r.packed[k].codes) and torch.equal(q.exps, r.packed[k].exps), k
    args = (rows["dz"], rows["dh"], rows["y"], rows["u"], rows["z"])
    got = nb.backward(*args, p, off)
    ref, size = R.norm_backward(*(wide(t) for t in args), v, o, kind, gate, 1e-5)
    check_backward(nb, got, ref, size, dtype, max(sizes))
    again = nb.backward(*args, p, off)
    assert torch.equal(again.dx, got.dx) and torch.equal(again.params.post_weight, got.params.post_weight)
    # from 8 bits: the formula at the values that the checkpoints stand for, one of them left plain
    q = [mt.pack8(t) if t is not None else None for t in (rows["y"], rows["u"], rows["z"])]
    seen = [R.unpack(t.codes.cpu().numpy(), t.exps.cpu().numpy()) if t is not None else None for t in q]
    ref, size = R.norm_backward(wide(rows["dz"]), wide(rows["dh"]), *seen, v, o, kind, gate, 1e-5)
    check_backward(nb, nb.backward(rows["dz"], rows["dh"], *q, p, off), ref, size, dtype, max(sizes))
    ref, size = R.norm_backward(wide(rows["dz"]), wide(rows["dh"]), seen[0], seen[1], wide(rows["z"]), v, o, kind, gate, 1e-5)
    check_backward(nb, nb.backward(rows["dz"], rows["dh"], q[0], q[1], rows["z"], p, off), ref, size, dtype, max(sizes))
    assert nb.error() == 0


@pytest.mark.parametrize("d", [4096, 5000, 8192])
def test_norm_wide_rows(d):
    rows, p, off = norm_case(12, [5, 7], 0, 1, d, "bf16", "silu")
    nb = mt.GatedNorm(d, num_groups=2, kind="layer")
    r = nb.forward(rows["x"], rows["y"], rows["u"], p, off, pack="h")
    z, h = R.norm_forward(wide(rows["x"]), wide(rows["y"]), wide(rows["u"]), values(p), wide(off), "layer", "silu", 1e-6)
    near(r.z, z, 4 * row_tol(z, "f32") + 2.0 ** -8 * np.abs(z))
    near(r.h, h, 4 * row_tol(h, "f32") + 2.0 ** -8 * np.abs(h))
    q = mt.pack8(r.h)
    assert torch.equal(q.codes, r.packed["h"].codes) and torch.equal(q.exps, r.packed["h"].exps)
    args = (rows["dz"], rows["dh"], rows["y"], rows["u"], rows["z"])
    ref, size = R.norm_backward(*(wide(t) for t in args), values(p), wide(off), "layer", "silu", 1e-6)
    check_backward(nb, nb.backward(*args, p, off), ref, size, "bf16", 7)


@pytest.mark.parametrize("d", [64, 96])
def test_norm_many_rows(d):
    """More rows than one chunk per block, groups that end inside a block's rows."""
    rows, p, off = norm_case(13, [9000, 1, 0, 12345], 10, 20, d, "bf16", "silu")
    nb = mt.GatedNorm(d, num_groups=4)
    args = (rows["dz"], rows["dh"], rows["y"], rows["u"], rows["z"])
    ref, size = R.norm_backward(*(wide(t) for t in args), values(p), wide(off), "rms", "silu", 1e-6)
    check_backward(nb, nb.backward(*args, p, off), ref, size, "bf16", 12345)


def test_norm_parts():
    """Only the norm before a block; only the norm after it; one group without offsets; [dim] parameters."""
    rows, p, off = norm_case(14, [40], 0, 0, 96, "f32", "silu")
    v, o = values(p), wide(off)
    nb = mt.GatedNorm(96, kind="layer", dtype="f32")
    first = mt.NormParams(pre_weight=p.pre_weight[0], pre_bias=p.pre_bias[0])
    r = nb.forward(rows["x"], params=first, pack="zh")
    assert r.z is rows["x"]
    only = {k: (v[k] if k.startswith("pre") else None) for k in v}
    _, h = R.norm_forward(wide(rows["x"]), None, None, only, o, "layer", "silu", 1e-6)
    near(r.h, h, 4 * row_tol(h, "f32"))
    q = mt.pack8(rows["x"])
    assert torch.equal(q.codes, r.packed["z"].codes)
    got = nb.backward(None, rows["dh"], z=r.packed["z"], params=first)
    ref, size = R.norm_backward(None, wide(rows["dh"]), None, None, R.unpack(q.codes.cpu().numpy(), q.exps.cpu().numpy()), only, o, "layer", "silu", 1e-6)
    near(got.dx, ref["dx"], 4 * row_tol(ref["dx"], "f32"))
    assert got.dy is None and got.du is None and got.params.post_weight is None
    near(got.params.pre_weight, ref["pre_weight"], 80 * F * (size["pre_weight"] + 1e-6))
    last = mt.NormParams(post_weight=p.post_weight, scale=p.scale)
    r = nb.forward(rows["x"], rows["y"], rows["u"], last)
    assert r.h is None
    only = {k: (v[k] if k in ("post_weight", "scale") else None) for k in v}
    z, _ = R.norm_forward(wide(rows["x"]), wide(rows["y"]), wide(rows["u"]), only, o, "layer", "silu", 1e-6)
    near(r.z, z, 4 * row_tol(z, "f32"))
    got = nb.backward(rows["dz"], None, rows["y"], rows["u"], params=last)
    ref, size = R.norm_backward(wide(rows["dz"]), None, wide(rows["y"]), wide(rows["u"]), None, only, o, "layer", "silu", 1e-6)
    check_backward(nb, got, ref, size, "f32", 40)


def test_norm_strided_and_unaligned():
    """y and u side by side in one product's output, their gradients side by side in one tensor."""
    for lo in (0, 3):
        d = 64
        rows, p, off = norm_case(15, [33, 20], 0, 0, d, "bf16", "silu")
        wide_t = torch.zeros(53, 2 * d + lo, device=DEV, dtype=torch.bfloat16)
        y, u = wide_t[:, lo:lo + d], wide_t[:, lo + d:]
        y.copy_(rows["y"])
        u.copy_(rows["u"])
        nb = mt.GatedNorm(d, num_groups=2)
        a = nb.forward(rows["x"], rows["y"], rows["u"], p, off, pack="yu")
        b = nb.forward(rows["x"], y, u, p, off, pack="yu")
        assert torch.equal(a.z, b.z) and torch.equal(a.h, b.h) and torch.equal(a.packed["u"].codes, b.packed["u"].codes)
        grads = torch.full((53, 2 * d + lo), 9.0, device=DEV, dtype=torch.bfloat16)
        ga = nb.backward(rows["dz"], rows["dh"], rows["y"], rows["u"], rows["z"], p, off)
        gb = nb.backward(rows["dz"], rows["dh"], y, u, rows["z"], p, off, out_dy=grads[:, lo:lo + d], out_du=grads[:, lo + d:])
        assert torch.equal(ga.dy, gb.dy) and torch.equal(ga.du, grads[:, lo + d:]) and (grads[:, :lo] == 9).all()
        assert torch.equal(ga.params.scale, gb.params.scale)


def test_norm_gradients_against_differences():
    """Every gradient in a random direction against central differences of <dz, z> + <dh, h> in 64 bits."""
    rows, p, off = norm_case(16, [9, 0, 14], 0, 0, 40, "f32", "silu")
    nb = mt.GatedNorm(40, num_groups=3, kind="layer", dtype="f32")
    fw = nb.forward(rows["x"], rows["y"], rows["u"], p, off)
    got = nb.backward(rows["dz"], rows["dh"], rows["y"], rows["u"], fw.z, p, off)
    v, o = values(p), wide(off)
    base = {"x": wide(rows["x"]), "y": wide(rows["y"]), "u": wide(rows["u"])}
    grads = {"x": got.dx, "y": got.dy, "u": got.du, **{k: getattr(got.params, k) for k in v}}
    rng = np.random.default_rng(1)
    for name, grad in grads.items():
        V = rng.standard_normal(grad.shape)
        step = 1e-4

        def loss(s):
            b = {k: t + (s * step * V if k == name else 0.0) for k, t in base.items()}
            q = {k: t + (s * step * V if k == name else 0.0) for k, t in v.items()}
            z, h = R.norm_forward(b["x"], b["y"], b["u"], q, o, "layer", "silu", 1e-6)
            return (wide(rows["dz"]) * z).sum() + (wide(rows["dh"]) * h).sum()

        diff = (loss(1) - loss(-1)) / (2 * step)
        # truncation step^2 * third derivative (order one per element) and fp32 rounding of the gradient
        assert abs((wide(grad) * V).sum() - diff) <= 2e-5 * (np.abs(wide(grad) * V).sum() + 1.0), name


def test_norm_not_a_number_stays_in_its_row():
    rows, p, off = norm_case(17, [20, 20], 0, 0, 64, "bf16", "silu")
    rows["y"][5, 3], rows["x"][21, 0], rows["u"][30, 1] = float("nan"), float("inf"), float("-inf")
    nb = mt.GatedNorm(64, num_groups=2)
    r = nb.forward(rows["x"], rows["y"], rows["u"], p, off)
    bad = torch.zeros(40, dtype=torch.bool, device=DEV)
    bad[[5, 21, 30]] = True
    assert torch.isfinite(r.h[~bad]).all() and torch.isfinite(r.z[~bad]).all()
    assert torch.isnan(r.h[5]).all() and torch.isnan(r.z[5]).all() and not torch.isfinite(r.z[21, 0])
    zero = torch.zeros(3, 64, device=DEV, dtype=torch.bfloat16)
    one = mt.NormParams(pre_weight=torch.ones(64, device=DEV))
    assert not mt.GatedNorm(64).forward(zero, params=one).h.any()  # a row of zeros divides by sqrt(eps)


@pytest.mark.parametrize("bad", [[0, 40, 20, 100], [-5, 10, 50, 4000]])
def test_norm_bad_offsets_latch(bad):
    rows, p, _ = norm_case(18, [30, 30, 40], 0, 0, 64, "bf16", "silu")
    off = torch.tensor(bad, dtype=torch.int64, device=DEV)
    nb = mt.GatedNorm(64, num_groups=3)
    r = nb.forward(rows["x"], rows["y"], rows["u"], p, off)
    z, _ = R.norm_forward(wide(rows["x"]), wide(rows["y"]), wide(rows["u"]), values(p), R.safe_offsets(bad, 100), "rms", "silu", 1e-6)
    near(r.z, z, 4 * row_tol(z, "f32") + 2.0 ** -8 * np.abs(z))
    args = (rows["dz"], rows["dh"], rows["y"], rows["u"], rows["z"])
    ref, size = R.norm_backward(*(wide(t) for t in args), values(p), R.safe_offsets(bad, 100), "rms", "silu", 1e-6)
    check_backward(nb, nb.backward(*args, p, off), ref, size, "bf16", 100)
    assert nb.error(clear=True) == mt.MT_EINVAL


def test_empty_batch():
    nb = mt.GatedNorm(64, num_groups=2)
    e = torch.empty(0, 64, device=DEV, dtype=torch.bfloat16)
    p = mt.NormParams(post_weight=torch.ones(2, 64, device=DEV), pre_weight=torch.ones(2, 64, device=DEV))
    off = torch.zeros(3, dtype=torch.int64, device=DEV)
    r = nb.forward(e, e, e, p, off, pack="h")
    assert r.z.shape == (0, 64) and r.h.shape == (0, 64) and r.packed["h"].shape == (0, 64)
    g = nb.backward(e, e, e, e, e, p, off)
    assert g.dx.shape == (0, 64) and not g.params.post_weight.any() and not g.params.pre_weight.any()
    assert mt.unpack8(mt.pack8(e)).shape == (0, 64)


def test_rows_past_32_bit_offsets():
    """2.2e9 values: the last rows come out as they do on their own (elements, codes and exponents past 2^31)."""
    n, d, tail = 4_300_000, 512, 300
    x = torch.empty(n, d, device=DEV, dtype=torch.bfloat16).normal_(generator=torch.Generator(device=DEV).manual_seed(23))
    last = x[-tail:].clone()
    p, q = mt.pack8(x), mt.pack8(last)
    assert torch.equal(p.codes[-tail:], q.codes) and torch.equal(p.exps[-tail:], q.exps)
    assert torch.equal(mt.unpack8(p)[-tail:], mt.unpack8(q))
    w = rand(torch.Generator(device=DEV).manual_seed(24), 2, 64, d, scale=d ** -0.5)
    off, alone = offsets_of([n - 200, 200]), offsets_of([100, 200])
    lin = mt.GroupedLinear(2, d, 64)
    assert torch.equal(lin.forward(x, w, off)[-tail:], lin.forward(last, w, alone))
    dy = torch.zeros(n, 64, device=DEV, dtype=torch.bfloat16)
    dy[-200:] = rand(torch.Generator(device=DEV).manual_seed(25), 200, 64)
    for saved, near_by in ((x, last), (p, q)):
        dx, dw = lin.backward(dy, saved, w, off)
        sdx, sdw = lin.backward(dy[-tail:], near_by, w, alone)
        assert torch.equal(dx[-tail:], sdx)
        near(dw[1], wide(sdw[1]), 216 * F * np.abs(wide(sdw[1])).max())
        assert not dw[0].any()
    nb = mt.GatedNorm(d, num_groups=2, kind="layer")
    one = mt.NormParams(pre_weight=torch.ones(2, d, device=DEV))
    assert torch.equal(nb.forward(x, params=one, offsets=off).h[-tail:], nb.forward(last, params=one, offsets=alone).h)
    g = nb.backward(None, x, z=p, params=one, offsets=off)
    assert torch.equal(g.dx[-tail:], nb.backward(None, last, z=q, params=one, offsets=alone).dx)


# ---- streams, graphs, refusals -----------------------------------------------------------------------------------------

def test_other_streams_and_graph_capture():
    """Calls on a given stream match the current stream's, and a captured forward and backward replay."""
    x, w, dy, off = linear_case(21, [500, 300], 0, 0, "bf16", 64, 128)
    rows, p, noff = norm_case(22, [500, 300], 0, 0, 128, "bf16", "silu")
    lin, nb = mt.GroupedLinear(2, 64, 128), mt.GatedNorm(128, num_groups=2)

    def step(stream=None):
        y = lin.forward(x, w, off, stream=stream)
        r = nb.forward(rows["x"], y, rows["u"], p, noff, pack="h", stream=stream)
        g = nb.backward(rows["dz"], rows["dh"], y, rows["u"], r.z, p, noff, stream=stream)
        dx, dw = lin.backward(g.dy, x, w, off, stream=stream)
        return [y, r.z, r.h, r.packed["h"].codes, g.dx, g.params.scale, dx, dw]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph_stream = torch.cuda.Stream()
    lin.reserve_workspace(800, stream=graph_stream)
    nb.reserve_workspace(800, stream=graph_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=graph_stream):
        held = step()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_refusals():
    t = dict(device=DEV, dtype=torch.bfloat16)
    lin = mt.GroupedLinear(2, 16, 24)
    x, w, off = torch.zeros(10, 16, **t), torch.zeros(2, 24, 16, **t), offsets_of([4, 6])
    for bad in (dict(x=x.float()), dict(x=x[:, :8]), dict(x=x.cpu()), dict(x=torch.zeros(16, 10, **t).t()), dict(x=x[0]),
                dict(weight=w.float()), dict(weight=w[:, :, :8]), dict(weight=w.transpose(1, 2)), dict(offsets=off.int()),
                dict(offsets=off[:2]), dict(offsets=off.cpu()), dict(offsets=[0, 4, 10]), dict(out=torch.zeros(9, 24, **t)),
                dict(x=x[:1].expand(10, 16))):
        with pytest.raises((TypeError, ValueError)):
            lin.forward(**{**dict(x=x, weight=w, offsets=off), **bad})
    dy = torch.zeros(10, 24, **t)
    for bad in (dict(x=None), dict(x=x[:5]), dict(x=mt.pack8(x[:5])), dict(dy=dy[:, :16]), dict(want_dx=False, want_dw=False),
                dict(out_dw=torch.zeros(2, 24, 16, **t))):
        with pytest.raises((TypeError, ValueError)):
            lin.backward(**{**dict(dy=dy, x=x, weight=w, offsets=off), **bad})
    for args in ((0, 16, 24), (1025, 16, 24), (2, 0, 24), (2, 16, 9000)):
        with pytest.raises(mt.MTError):
            mt.GroupedLinear(*args)
    with pytest.raises(ValueError):
        mt.GroupedLinear(2, 16, 24, dtype="f16")
    nb = mt.GatedNorm(16)
    p = mt.NormParams(post_weight=torch.ones(1, 16, device=DEV), pre_weight=torch.ones(16, device=DEV))
    for bad in (dict(y=None), dict(u=None), dict(params=mt.NormParams()), dict(pack="q"), dict(x=x.float()), dict(y=x[:5]),
                dict(params=mt.NormParams(post_weight=torch.ones(2, 16, device=DEV))), dict(offsets=off),
                dict(params=mt.NormParams(post_weight=torch.ones(1, 16, **t))),
                dict(params=mt.NormParams(post_weight=p.post_weight, pre_bias=p.pre_weight))):
        with pytest.raises((TypeError, ValueError)):
            nb.forward(**{**dict(x=x, y=x, u=x, params=p), **bad})
    with pytest.raises(ValueError):
        nb.backward(x, x, x, x, None, p)
    with pytest.raises(ValueError):
        nb.backward(x, None, x, x, x, p)
    with pytest.raises(ValueError):
        mt.GatedNorm(16, num_groups=2).forward(x, params=mt.NormParams(pre_weight=torch.ones(2, 16, device=DEV)))
    for kw in (dict(eps=0.0), dict(dim=0), dict(dim=9000), dict(num_groups=0)):
        with pytest.raises(mt.MTError):
            mt.GatedNorm(**{**dict(dim=16), **kw})
    with pytest.raises(ValueError):
        mt.GatedNorm(16, kind="batch")
    with pytest.raises(TypeError):
        mt.pack8(x.half())
    with pytest.raises(ValueError):
        mt.pack8(torch.zeros(2, 9000, **t))
    with pytest.raises(ValueError):
        mt.Packed8(torch.zeros(4, 33, device=DEV, dtype=torch.int8), torch.zeros(4, 1, device=DEV, dtype=torch.uint8))


def test_example_trains_through_the_table():
    """Lookup, tower, gradients from 8-bit checkpoints, sparse Adam: the loss falls; serving takes the same weights."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import dense_block
    losses = dense_block.train(steps=25, users=24, width=64, verbose=False)
    assert all(np.isfinite(losses)) and np.mean(losses[-5:]) < 0.9 * np.mean(losses[:5]), losses

"""The gated feed-forward part against its 64-bit definition.

Tolerances, from the arithmetic:
* a product of k values is at most (k + 64) 2^-23 of the sum of the absolute products off (a tensor core may cut off where an
  fp32 add rounds; three bf16 parts of an fp32 value leave out less than 2^-24 of a product);
* a gate and its derivative go through an exponential and a reciprocal (2^-22 each) and a few roundings: 2^-19 of the larger
  of the gate's factor and |u|, and they follow u's error by their derivative;
* a bf16 value is rounded by at most 2^-8 of it, fp32 2^-24: h once; the gradients of y and u once, and dx and dw once more.
"""
import pytest
import torch

import loss_reference as R
import update_merged_table_gb300 as mt

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
F = 2.0 ** -23
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def near(got, want, tol, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist(),
                                 tol.expand_as(want)[bad][:4].tolist())


def offsets_of(sizes, lead=0):
    o = [lead]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int64, device=DEV)


def make(seed, sizes, lead, tail, dtype, k, m):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = lead + sum(sizes) + tail

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(TORCH[dtype])

    return rand(n, k), rand(len(sizes), 2 * m, k, scale=k ** -0.5), rand(n, m), offsets_of(sizes, lead)


def checked(got, what, ref, dtype, gate, k, dh=None):
    """Holds h, or (dx, dw), to the reference."""
    half = HALF[dtype]
    ey, eu = (k + 64) * F * ref["sy"], (k + 64) * F * ref["su"]
    act, dact, second = R.gate(ref["u"], gate)
    size = torch.maximum(act.abs(), ref["u"].abs()) + 1.0
    ea, eda = dact.abs() * eu + second * eu * eu + 2.0 ** -19 * size, second * eu + 2.0 ** -19 * size
    if what == "h":
        near(got, ref["h"], half * ref["h"].abs() + (1 + 2 * half) * (ey * act.abs() + (ref["y"].abs() + ey) * ea) + 1e-38, what)
        return
    edy = dh.abs() * ea
    edu = dh.abs() * (ey * (dact.abs() + eda) + ref["y"].abs() * eda)
    edy, edu = edy + 1.01 * half * (ref["dy"].abs() + edy), edu + 1.01 * half * (ref["du"].abs() + edu)
    return edy, edu


def check_all(x, w, dh, off, dtype, gate, lin=None, h=None, grads=None):
    k, m = x.shape[1], dh.shape[1]
    lin = lin or mt.GatedLinear(w.shape[0], k, m, gate=gate, dtype=dtype)
    h = lin.forward(x, w, off) if h is None else h
    X, W, D = x.double(), w.double(), dh.double()
    ref = R.gated(X, W, off, gate, D)
    checked(h, "h", ref, dtype, gate, k)
    dx, dw = lin.backward(dh, x, w, off) if grads is None else grads
    edy, edu = checked(None, "d", ref, dtype, gate, k, D)
    e = torch.cat([edy, edu], 1)
    half = HALF[dtype]
    tdx, tdw = torch.zeros_like(X), torch.zeros_like(W)
    for g, (a, b) in enumerate(R.spans(off)):
        tdx[a:b] = e[a:b] @ W[g].abs()
        tdw[g] = e[a:b].T @ X[a:b].abs()
    longest = max([b - a for a, b in R.spans(off)])
    near(dx, ref["dx"], half * ref["dx"].abs() + 1.01 * tdx + (2 * m + 64) * F * ref["sdx"] + 1e-38, "dx")
    near(dw, ref["dw"], half * ref["dw"].abs() + 1.01 * tdw + (longest + 64) * F * ref["sdw"] + 1e-38, "dw")
    assert lin.error() == 0
    return lin, h, (dx, dw)


SIZES = [
    ([1], 0, 0),
    ([0, 5, 0, 130, 1], 0, 0),
    ([0, 0], 3, 2),              # no row in any group
    ([257, 0, 129, 300], 2, 3),  # rows before and after the groups
    ([3] * 61, 0, 0),
]


@pytest.mark.parametrize("sizes,lead,tail", SIZES)
@pytest.mark.parametrize("dtype,k,m", [("bf16", 64, 128), ("bf16", 8, 8), ("bf16", 72, 200), ("bf16", 50, 33), ("bf16", 1, 1),
                                       ("bf16", 192, 129), ("f32", 16, 64), ("f32", 50, 33), ("f32", 130, 200), ("f32", 1, 1)])
def test_forward_and_gradients(sizes, lead, tail, dtype, k, m):
    x, w, dh, off = make(1, sizes, lead, tail, dtype, k, m)
    lin, h, (dx, dw) = check_all(x, w, dh, off, dtype, "silu")
    n, a, b = x.shape[0], int(off[0]), int(off[-1])
    assert not h[:a].any() and not h[b:].any() and not dx[:a].any() and not dx[b:].any()
    again = lin.backward(dh, x, w, off)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(lin.forward(x, w, off), h)


@pytest.mark.parametrize("gate", ["linear", "sigmoid", "silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates(gate, dtype):
    x, w, dh, off = make(2, [40, 77], 1, 1, dtype, 40, 56)
    x = x * 3  # gates far into both ends
    check_all(x, w, dh, off, dtype, gate)


@pytest.mark.parametrize("gate", ["linear", "sigmoid", "silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_gates(gate, dtype):
    """u of 1e20 to 1e22 either way: its square is no fp32 number, everything that is asked for is one."""
    x, w, dh, off = make(13, [40, 5], 0, 0, dtype, 24, 40)
    w[:, 40:] *= 1e21
    _, h, (dx, dw) = check_all(x, w, dh, off, dtype, gate)
    assert bool(torch.isfinite(h).all()) and bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("sizes,k,m", [([9001, 0, 3, 20000], 256, 512), ([300, 700, 40], 1024, 2048), ([129, 2], 2048, 1032),
                                       ([2000] * 8, 512, 1024), ([6000, 5001], 33, 250)])
def test_long_groups(sizes, k, m):
    """Several tiles in every direction, pairs of blocks, and groups whose dw comes in several parts."""
    x, w, dh, off = make(3, sizes, 5, 7, "bf16", k, m)
    check_all(x, w, dh, off, "bf16", "silu")


def test_widest():
    x, w, dh, off = make(4, [70], 0, 0, "bf16", 16, 8192)
    check_all(x, w, dh, off, "bf16", "silu")
    x, w, dh, off = make(5, [70], 0, 0, "bf16", 8192, 24)
    check_all(x, w, dh, off, "bf16", "silu")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_rows_and_outputs(dtype):
    gen = torch.Generator(device=DEV).manual_seed(6)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(TORCH[dtype])

    for lo in (0, 8, 3):
        k, m = 64, 96
        big_x, big_dh = rand(160, 200), rand(160, 300)
        x, dh = big_x[:, lo:lo + k], big_dh[:, lo:lo + m]
        w, off = rand(2, 2 * m, k) * k ** -0.5, offsets_of([100, 60])
        lin = mt.GatedLinear(2, k, m, dtype=dtype)
        big_h, big_dx = torch.full((160, 128), 7.0, device=DEV, dtype=TORCH[dtype]), torch.full((160, 80), 7.0, device=DEV, dtype=TORCH[dtype])
        out_dw = torch.empty(2, 2 * m, k, device=DEV, dtype=TORCH[dtype])
        lin.forward(x, w, off, out=big_h[:, lo:lo + m])
        grads = lin.backward(dh, x, w, off, out_dx=big_dx[:, lo:lo + k], out_dw=out_dw)
        assert grads[1].data_ptr() == out_dw.data_ptr()
        check_all(x, w, dh, off, dtype, "silu", lin, big_h[:, lo:lo + m], grads)
        assert (big_h[:, :lo] == 7).all() and (big_h[:, lo + m:] == 7).all()
        assert (big_dx[:, :lo] == 7).all() and (big_dx[:, lo + k:] == 7).all()


@pytest.mark.parametrize("dtype,k,m", [("bf16", 64, 128), ("bf16", 50, 33), ("f32", 64, 128)])
def test_outputs_on_one_element(dtype, k, m):
    """Outputs that start on one element only, with rows of several parts of dw."""
    x, w, dh, off = make(14, [700, 0, 90], 2, 3, dtype, k, m)
    lin, h, (dx, dw) = check_all(x, w, dh, off, dtype, "silu")
    flat = [torch.full((t.numel() + 2,), 7.0, device=DEV, dtype=TORCH[dtype]) for t in (h, dx, dw)]
    out = [f[1:-1].view(t.shape) for f, t in zip(flat, (h, dx, dw))]
    assert torch.equal(lin.forward(x, w, off, out=out[0]), h)
    got = lin.backward(dh, x, w, off, out_dx=out[1], out_dw=out[2])
    check_all(x, w, dh, off, dtype, "silu", lin=lin, h=out[0], grads=got)  # (dx by the fp32 pipes: not the same bits)
    assert all(float(f[0]) == 7 and float(f[-1]) == 7 for f in flat)


def test_single_gradients_and_empty_batches():
    x, w, dh, off = make(7, [30, 50], 0, 0, "bf16", 64, 64)
    lin = mt.GatedLinear(2, 64, 64)
    dx, dw = lin.backward(dh, x, w, off)
    a, none = lin.backward(dh, x, w, off, want_dw=False)
    assert none is None and torch.equal(a, dx)
    none, b = lin.backward(dh, x, w, off, want_dx=False)
    assert none is None and torch.equal(b, dw)
    zero = torch.zeros(3, dtype=torch.int64, device=DEV)
    assert lin.forward(x[:0], w, zero).shape == (0, 64)
    dx, dw = lin.backward(dh[:0], x[:0], w, zero)
    assert dx.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_that_are_not_finite_stay_in_their_rows_and_groups(dtype):
    x, w, dh, off = make(8, [70, 130, 20], 2, 3, dtype, 72, 136)
    lin = mt.GatedLinear(3, 72, 136, dtype=dtype)
    h, (dx, dw) = lin.forward(x, w, off), lin.backward(dh, x, w, off)
    bad = x.clone()
    bad[1], bad[-1] = float("nan"), float("inf")  # in no group
    bad[75] = float("inf")                        # in group 1
    h2, (dx2, dw2) = lin.forward(bad, w, off), lin.backward(dh, bad, w, off)
    keep = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    keep[75] = False
    assert torch.equal(h2[keep], h[keep]) and torch.equal(dx2[keep], dx[keep])
    assert torch.equal(dw2[[0, 2]], dw[[0, 2]])


def test_bad_offsets_are_latched():
    x, w, dh, off = make(9, [30, 50], 0, 0, "bf16", 64, 64)
    lin = mt.GatedLinear(2, 64, 64)
    bad = torch.tensor([10, -5, 200], dtype=torch.int64, device=DEV)  # counts as [10, 10, 80]
    h = lin.forward(x, w, bad)
    safe = torch.tensor([10, 10, 80], dtype=torch.int64, device=DEV)
    assert lin.error(clear=True) == mt.MT_EINVAL
    assert torch.equal(h, lin.forward(x, w, safe)) and lin.error() == 0


def test_gradients_against_differences():
    """fp32, along random directions; differences of a 64-bit loss of the library's own outputs."""
    x, w, dh, off = make(10, [20, 13], 1, 2, "f32", 24, 40)
    for gate in ("sigmoid", "silu", "gelu"):
        lin = mt.GatedLinear(2, 24, 40, gate=gate, dtype="f32")
        dx, dw = lin.backward(dh, x, w, off)
        gen = torch.Generator(device=DEV).manual_seed(11)
        for what, grad in (("x", dx), ("w", dw)):
            v = torch.randn(grad.shape, generator=gen, device=DEV)
            out, step = [], 2.0 ** -7
            for s in (step, -step):
                h = lin.forward(x + s * v if what == "x" else x, w + s * v if what == "w" else w, off)
                out.append((dh.double() * h.double()).sum())
            diff = (out[0] - out[1]) / (2 * step)
            # the third derivative's part, step^2 / 6 of it, and rounding of h over the step
            size = float((grad.double() * v.double()).abs().sum())
            assert abs(float(diff) - float((grad.double() * v.double()).sum())) <= 2e-3 * size, (gate, what)


def test_streams_and_graphs():
    x, w, dh, off = make(12, [300, 500], 0, 0, "bf16", 128, 192)
    lin = mt.GatedLinear(2, 128, 192)
    h, (dx, dw) = lin.forward(x, w, off), lin.backward(dh, x, w, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h2, g2 = lin.forward(x, w, off, stream=s), lin.backward(dh, x, w, off, stream=s)
    s.synchronize()
    assert torch.equal(h2, h) and torch.equal(g2[0], dx) and torch.equal(g2[1], dw)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = lin.forward(x, w, off), lin.backward(dh, x, w, off)
        graphs.append((g, o))
    for g, (gh, gg) in graphs:  # side by side
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            g.replay()
    lin.backward(dh, x, w, off)
    torch.cuda.synchronize()
    for _, (gh, gg) in graphs:
        assert torch.equal(gh, h) and torch.equal(gg[0], dx) and torch.equal(gg[1], dw)


def test_refusals():
    x, w, dh, off = make(13, [30, 50], 0, 0, "bf16", 64, 64)
    lin = mt.GatedLinear(2, 64, 64)
    for bad in (dict(num_groups=0), dict(in_dim=8193), dict(out_dim=0), dict(out_dim=8193)):
        with pytest.raises(mt.MTError):
            mt.GatedLinear(**{**dict(num_groups=2, in_dim=64, out_dim=64), **bad})
    with pytest.raises(ValueError):
        mt.GatedLinear(2, 64, 64, gate="none")
    with pytest.raises(TypeError):
        lin.forward(x.float(), w, off)
    with pytest.raises(ValueError):
        lin.forward(x, w[:, :64], off)
    with pytest.raises(ValueError):
        lin.forward(x[:, ::2], w, off)
    with pytest.raises(TypeError):
        lin.forward(x, w, off.int())
    with pytest.raises(ValueError):
        lin.backward(dh[:-1], x, w, off)
    with pytest.raises(ValueError):
        lin.backward(dh, x, w, off, want_dx=False, want_dw=False)
    with pytest.raises(mt.MTError):
        lin.forward(x, w, off, out=x)  # the output would overlap the input
    with pytest.raises(mt.MTError):
        lin.backward(dh, x, w, off, out_dx=x)
    with pytest.raises(ValueError):
        lin.backward(dh, x, w, off, out_dw=torch.empty(2, 128, 64, device=DEV))

"""Cross entropy and distillation over a vocabulary against their 64-bit definitions.

Tolerances, from the arithmetic (all of a row's logits z, of the sizes sz = scale * sum |x w|):
* a logit is ez = (dim + 64) 2^-23 max sz off, and a few 2^-24 of itself more when it is scaled and taken to base 2;
* an exponential is 2^-22 off, a sum of them by as many roundings as adds follow one another: under vocab / 32 + 64;
  lse then by ez + 2^-20 + (vocab / 32 + 64) 2^-24 + 2^-22 max |z| and its own rounding 2^-24 |lse|;
* a loss adds up lse, the shares' logits and the mean logit: four such errors and (top + 8) 2^-23 of the sizes;
* p = exp(z - lse) is e = 2 (what lse is off) + 2^-20 of itself off; dz is a few roundings more, and with bf16 rows rounded
  by 2^-8 of itself; the products of dz add k 2^-23 of the sum of their sizes, and the result is rounded once.
"""
import math

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


def make(seed, n, v, d, dtype, top=0, masked=0.3, spread=1.5):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=DEV) * scale

    w = rand(v, d, scale=spread * d ** -0.5)
    hit = torch.randint(0, v, (n,), generator=gen, device=DEV)
    s = {"x": (rand(n, d) + w[hit]).to(TORCH[dtype]), "w": w.to(TORCH[dtype]), "dloss": rand(n) / n}
    out = torch.rand(n, generator=gen, device=DEV) < masked
    if top == 0:
        s["targets"] = torch.where(out, -1, hit).to(torch.int32)
    else:
        ids = torch.randint(0, v, (n, top), generator=gen, device=DEV)
        ids = torch.where(torch.rand(n, top, generator=gen, device=DEV) < 0.2, -1, ids)
        s["ids"] = torch.where(out[:, None], -1, ids).to(torch.int32)
        s["logits"] = rand(n, top, scale=2.0)
    return s


def given(s):
    return (s["targets"],) if "targets" in s else (s["ids"], s["logits"])


def check_all(s, dtype, scale=1.0, smoothing=0.0, z_loss=0.0, handle=None, forward=None, grads=None):
    n, d = s["x"].shape
    v = s["w"].shape[0]
    if handle is None:
        handle = mt.CrossEntropy(v, d, scale=scale, smoothing=smoothing, z_loss=z_loss, dtype=dtype) if "targets" in s \
            else mt.Distillation(v, d, s["ids"].shape[1], scale=scale, dtype=dtype)
    r = handle.forward(s["x"], s["w"], *given(s)) if forward is None else forward
    dx, dw = handle.backward(s["dloss"], s["x"], s["w"], *given(s), r.lse) if grads is None else grads
    X, W = s["x"].double(), s["w"].double()
    more = dict(targets=s["targets"], smoothing=smoothing, z_loss=z_loss) if "targets" in s else dict(ids=s["ids"], logits=s["logits"].double())
    ref = R.loss(X, W, scale, dloss=s["dloss"].double(), **more)
    big = ref["z"].abs().amax(1)
    ez = (d + 64) * F * ref["sz"].amax(1) + 4 * 2.0 ** -24 * big
    e = ez + 2.0 ** -20 + (v / 32 + 64) * 2.0 ** -24 + 2.0 ** -22 * big
    near(r.lse, ref["lse"], torch.where(ref["live"], e + 2.0 ** -24 * ref["lse"].abs(), 0.0), "lse")
    top = s["ids"].shape[1] if "ids" in s else 1
    sizes = ref["lse"].abs() + big + z_loss * ref["lse"] ** 2 + math.log(top + 1)
    tol = (4 + 2 * z_loss * ref["lse"].abs()) * e + (top + 8) * F * sizes
    near(r.loss, ref["loss"], torch.where(ref["live"], tol, 0.0), "loss")
    half = HALF[dtype]
    g = s["dloss"].double().abs()[:, None] * scale
    # what the parts of dz are off, each by its own size
    parts = g * torch.where(ref["live"][:, None], ref["p"] * (1 + 2 * z_loss * ref["lse"].abs())[:, None] * (2 * e + 2.0 ** -20)[:, None]
                            + 4 * 2.0 ** -24 * (ref["p"] + smoothing / v), 0.0)
    if "targets" in s:
        at, t = s["targets"].long().clamp(min=0)[:, None], ref["live"].double()[:, None]
    else:
        t, at, _ = R.shares(s["ids"], s["logits"].double(), scale, v)
    # a share is a softmax over top pairs in fp32: (top + 16) roundings
    parts.scatter_add_(1, at, g * t * (top + 16) * 2.0 ** -22)
    parts = parts + 1.01 * half * (ref["dz"].abs() + parts)
    x = torch.where(ref["live"][:, None], X, 0.0)
    near(dx, ref["dx"], half * ref["dx"].abs() + 1.01 * (parts @ W.abs()) + (v + 64) * F * ref["sdx"] + 1e-38, "dx")
    near(dw, ref["dw"], half * ref["dw"].abs() + 1.01 * (parts.T @ x.abs()) + (n + 64) * F * ref["sdw"] + 1e-38, "dw")
    dead = ~ref["live"]
    assert not r.loss[dead].any() and not r.lse[dead].any() and not dx[dead].any()
    return handle, r, (dx, dw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,d", [(1, 1, 1), (1, 2, 8), (2, 255, 64), (37, 256, 20), (128, 257, 72), (129, 1000, 130), (300, 513, 264),
                                   (65, 5003, 16), (5, 30000, 40), (1000, 7, 512)])
def test_cross_entropy(n, v, d, dtype):
    s = make(1, n, v, d, dtype)
    handle, r, (dx, dw) = check_all(s, dtype)
    again = handle.forward(s["x"], s["w"], s["targets"])
    assert torch.equal(again.loss, r.loss) and torch.equal(again.lse, r.lse)
    ax, aw = handle.backward(s["dloss"], s["x"], s["w"], s["targets"], r.lse)
    assert torch.equal(ax, dx) and torch.equal(aw, dw)
    assert handle.error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,d,top", [(1, 1, 1, 1), (3, 2, 8, 5), (37, 256, 20, 8), (129, 1000, 130, 33), (70, 513, 264, 100), (20, 5003, 16, 1024)])
def test_distillation(n, v, d, top, dtype):
    s = make(2, n, v, d, dtype, top=top)
    check_all(s, dtype)
    check_all({**s, "ids": s["ids"].long(), "logits": s["logits"].bfloat16()}, dtype, scale=0.25)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,smoothing,z_loss", [(2.0, 0.0, 0.0), (1.0, 0.1, 0.0), (0.5, 0.0, 1e-2), (1.5, 0.3, 1e-3)])
def test_scale_smoothing_and_z_loss(scale, smoothing, z_loss, dtype):
    check_all(make(3, 100, 700, 96, dtype), dtype, scale, smoothing, z_loss)


@pytest.mark.parametrize("n,v,d,top", [(2048, 20000, 256, 0), (4096, 5000, 512, 0), (2048, 20000, 256, 16), (65537, 4500, 16, 0), (3, 100003, 256, 0),
                                       (20000, 300, 64, 0), (5000, 30000, 200, 0), (700, 40000, 130, 3), (20000, 2500, 100, 0), (9000, 9000, 264, 0)])
def test_long(n, v, d, top):
    """Pairs of blocks, vocabularies in several pieces and runs, few rows and few entries."""
    check_all(make(4, n, v, d, "bf16", top=top), "bf16")


@pytest.mark.parametrize("n,v,d", [(9000, 700, 64), (300, 40000, 200), (30000, 6000, 24)])
def test_long_fp32(n, v, d):
    check_all(make(5, n, v, d, "f32"), "f32", smoothing=0.1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [0, 4])
def test_rows_that_take_no_part(dtype, top):
    """All of them; and ones that hold what is not finite."""
    s = make(6, 300, 600, 64, dtype, top=top, masked=0.5)
    handle, r, (dx, dw) = check_all(s, dtype)
    dead = s["targets"] < 0 if top == 0 else (s["ids"] < 0).all(1)
    x = s["x"].clone()
    x[dead] = float("nan")
    x[torch.nonzero(dead)[0]] = float("inf")
    lse, g = r.lse.clone(), s["dloss"].clone()
    lse[dead], g[dead] = float("nan"), float("inf")  # nothing of such a row is read
    r2 = handle.forward(x, s["w"], *given(s))
    assert torch.equal(r2.loss, r.loss) and torch.equal(r2.lse, r.lse)
    dx2, dw2 = handle.backward(g, x, s["w"], *given(s), lse)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    none = (torch.full_like(s["targets"], -1),) if top == 0 else (torch.full_like(s["ids"], -5), s["logits"])
    r3 = handle.forward(x, s["w"], *none)
    assert not r3.loss.any() and not r3.lse.any()
    dx3, dw3 = handle.backward(g, x, s["w"], *none, lse)
    assert not dx3.any() and not dw3.any()
    assert handle.error() == 0


def test_pairs_that_are_not_there():
    """Logits of -inf, rows of nothing else, the same id several times, one pair alone."""
    s = make(7, 6, 50, 32, "f32", top=4, masked=0.0)
    s["ids"] = torch.tensor([[3, 3, 3, 7], [1, 2, -1, 4], [9, 9, 9, 9], [5, -1, -1, -1], [8, 0, 49, 8], [-1, 6, 6, -1]], dtype=torch.int32, device=DEV)
    s["logits"][1, 0] = s["logits"][2, :] = -math.inf
    s["logits"][5, 1] = -math.inf
    _, r, (dx, dw) = check_all(s, "f32")
    assert float(r.loss[2]) == 0 and not dx[2].any()


def test_large_logits():
    """Logits far apart and far from zero: one entry has all, and the others' exponentials vanish."""
    for dtype in ("bf16", "f32"):
        s = make(8, 64, 300, 64, dtype, spread=60.0)
        check_all(s, dtype)
        check_all(s, dtype, scale=4.0)


def test_an_infinity_or_nan_in_a_row_that_takes_part_stays_there():
    s = make(9, 200, 300, 64, "bf16", masked=0.0)
    handle, r, (dx, _) = check_all(s, "bf16")
    x = s["x"].clone()
    x[17, 3] = float("nan")
    r2 = handle.forward(x, s["w"], s["targets"])
    keep = torch.arange(200, device=DEV) != 17
    assert torch.equal(r2.loss[keep], r.loss[keep]) and bool(torch.isnan(r2.loss[17]))
    dx2, dw2 = handle.backward(s["dloss"], x, s["w"], s["targets"], r2.lse)
    assert torch.equal(dx2[keep], dx[keep]) and bool(torch.isnan(dx2[17]).all()) and bool(torch.isnan(dw2).all())


def test_targets_outside_the_vocabulary_are_latched():
    s = make(10, 50, 40, 16, "bf16", masked=0.0)
    handle = mt.CrossEntropy(40, 16)
    bad = s["targets"].clone()
    bad[3], bad[4] = 40, 2 ** 31 - 1
    r = handle.forward(s["x"], s["w"], bad)
    assert handle.error(clear=True) == mt.MT_EINVAL
    safe = s["targets"].clone()
    safe[3:5] = -1
    want = handle.forward(s["x"], s["w"], safe)
    assert torch.equal(r.loss, want.loss) and handle.error() == 0
    far = safe.long()
    far[0] = 2 ** 40
    handle.forward(s["x"], s["w"], far)
    assert handle.error(clear=True) == mt.MT_EINVAL
    d = mt.Distillation(40, 16, 2)
    ids = torch.tensor([[1, 40]] * 50, dtype=torch.int64, device=DEV)
    d.forward(s["x"], s["w"], ids, torch.zeros(50, 2, device=DEV))
    assert d.error() == mt.MT_EINVAL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_rows_and_outputs(dtype):
    for lo in (0, 8, 3):
        s = make(11, 90, 70, 64, dtype)
        big_x, big_w = torch.zeros(90, 100, device=DEV, dtype=TORCH[dtype]), torch.zeros(70, 90, device=DEV, dtype=TORCH[dtype])
        big_x[:, lo:lo + 64], big_w[:, lo:lo + 64] = s["x"], s["w"]
        t = {**s, "x": big_x[:, lo:lo + 64], "w": big_w[:, lo:lo + 64]}
        handle = mt.CrossEntropy(70, 64, dtype=dtype)
        big_dx = torch.full((90, 100), 7.0, device=DEV, dtype=TORCH[dtype])
        out_dw = torch.empty(70, 64, device=DEV, dtype=TORCH[dtype])
        out = torch.empty(2, 90, device=DEV)
        r = handle.forward(t["x"], t["w"], t["targets"], out_loss=out[0], out_lse=out[1])
        grads = handle.backward(t["dloss"], t["x"], t["w"], t["targets"], r.lse, out_dx=big_dx[:, lo:lo + 64], out_dw=out_dw)
        check_all(t, dtype, handle=handle, forward=r, grads=grads)
        assert (big_dx[:, :lo] == 7).all() and (big_dx[:, lo + 64:] == 7).all()


@pytest.mark.parametrize("n,v,d,dtype", [(300, 600, 64, "bf16"), (300, 600, 200, "bf16"), (3000, 20000, 264, "bf16"), (300, 600, 72, "f32")])
def test_unaligned_outputs_and_no_row(n, v, d, dtype):
    """Gradients that start on one element only; then no row at all that takes part."""
    s = make(15, n, v, d, dtype)
    handle, r, (dx, dw) = check_all(s, dtype)
    flat = [torch.full((k * d + 2,), 7.0, device=DEV, dtype=TORCH[dtype]) for k in (n, v)]
    out = [f[1:-1].view(-1, d) for f in flat]
    got = handle.backward(s["dloss"], s["x"], s["w"], s["targets"], r.lse, out_dx=out[0], out_dw=out[1])
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    none = torch.full_like(s["targets"], -1)
    r = handle.forward(s["x"], s["w"], none)
    assert not r.loss.any() and not r.lse.any()
    got = handle.backward(s["dloss"], s["x"], s["w"], none, r.lse, out_dx=out[0], out_dw=out[1])
    assert not got[0].any() and not got[1].any()
    assert all(float(f[0]) == 7 and float(f[-1]) == 7 for f in flat) and handle.error() == 0


def test_single_gradients_and_empty_batches():
    s = make(12, 60, 90, 64, "bf16")
    handle, r, (dx, dw) = check_all(s, "bf16")
    a, none = handle.backward(s["dloss"], s["x"], s["w"], s["targets"], r.lse, want_dw=False)
    assert none is None and torch.equal(a, dx)
    none, b = handle.backward(s["dloss"], s["x"], s["w"], s["targets"], r.lse, want_dx=False)
    assert none is None and torch.equal(b, dw)
    e = handle.forward(s["x"][:0], s["w"], s["targets"][:0])
    assert e.loss.shape == (0,) and e.lse.shape == (0,)
    dx, dw = handle.backward(s["dloss"][:0], s["x"][:0], s["w"], s["targets"][:0], e.lse)
    assert dx.shape == (0, 64) and not dw.any()


def test_streams_and_graphs():
    s = make(13, 500, 3000, 128, "bf16", top=8)
    handle, r, (dx, dw) = check_all(s, "bf16")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    r2 = handle.forward(s["x"], s["w"], *given(s), stream=st)
    dx2, dw2 = handle.backward(s["dloss"], s["x"], s["w"], *given(s), r2.lse, stream=st)
    st.synchronize()
    assert torch.equal(r2.loss, r.loss) and torch.equal(dx2, dx) and torch.equal(dw2, dw)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gr = handle.forward(s["x"], s["w"], *given(s))
            out = gr.loss, *handle.backward(s["dloss"], s["x"], s["w"], *given(s), gr.lse)
        graphs.append((g, out))
    for g, _ in graphs:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            g.replay()
    handle.backward(s["dloss"], s["x"], s["w"], *given(s), r.lse)
    torch.cuda.synchronize()
    for _, out in graphs:
        for a, b in zip(out, (r.loss, dx, dw)):
            assert torch.equal(a, b)


def test_replayed_graphs_follow_their_inputs():
    """How many rows take part is found on the device: a replay with other targets in place is right too."""
    s = make(17, 300, 900, 64, "bf16", masked=0.2)
    handle = mt.CrossEntropy(900, 64)
    handle.forward(s["x"], s["w"], s["targets"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = handle.forward(s["x"], s["w"], s["targets"])
        dx, dw = handle.backward(s["dloss"], s["x"], s["w"], s["targets"], r.lse)
    for masked in (0.9, 0.0, 1.1):
        t = make(18 + int(10 * masked), 300, 900, 64, "bf16", masked=masked)
        for k in ("x", "w", "targets", "dloss"):
            s[k].copy_(t[k])
        g.replay()
        check_all(t, "bf16", handle=handle, forward=r, grads=(dx, dw))


def test_threads_and_streams_side_by_side():
    import threading
    cases = [make(20 + i, 400 + 100 * i, 2000 + 500 * i, 64 + 72 * i, "bf16", top=i) for i in range(4)]
    want, got = [], [None] * 4
    handles = [mt.CrossEntropy(s["w"].shape[0], s["x"].shape[1]) if "targets" in s else mt.Distillation(s["w"].shape[0], s["x"].shape[1], s["ids"].shape[1])
               for s in cases]
    for s, h in zip(cases, handles):
        r = h.forward(s["x"], s["w"], *given(s))
        want.append((r.loss, *h.backward(s["dloss"], s["x"], s["w"], *given(s), r.lse)))
    torch.cuda.synchronize()

    def work(i):
        st = torch.cuda.Stream()
        s, h = cases[i], handles[i]
        for _ in range(5):
            r = h.forward(s["x"], s["w"], *given(s), stream=st)
            g = h.backward(s["dloss"], s["x"], s["w"], *given(s), r.lse, stream=st)
        st.synchronize()
        got[i] = (r.loss, *g)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("n,v,d,dtype,top", [(70000, 40000, 136, "bf16", 0), (70000, 12001, 40, "f32", 0), (66001, 36000, 520, "bf16", 3)])
def test_vocabulary_in_pieces(n, v, d, dtype, top):
    """More of dz than there is room for: the vocabulary comes in two pieces (few rows take part)."""
    s = make(31, n, v, d, dtype, top=top, masked=0.99)
    live = (s["ids"] >= 0).any(1) if top else s["targets"] >= 0
    handle = mt.Distillation(v, d, top, dtype=dtype) if top else mt.CrossEntropy(v, d, dtype=dtype)
    args = (s["ids"], s["logits"]) if top else (s["targets"],)
    r = handle.forward(s["x"], s["w"], *args)
    dx, dw = handle.backward(s["dloss"], s["x"], s["w"], *args, r.lse)
    assert not r.loss[~live].any() and not r.lse[~live].any() and not dx[~live].any()
    c = {k: t if k == "w" else t[live] for k, t in s.items()}
    check_all(c, dtype, handle=handle, forward=mt.LossForward(r.loss[live], r.lse[live]), grads=(dx[live], dw))


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Rows of x, W and dx more than 2^31 elements apart from their first."""
    n, v, d, ld = 70000, 70000, 32, 40000
    s = make(30, n, v, d, "bf16", masked=0.98)  # (about 1400 rows take part: the last ones among them)
    s["targets"][-3:] = torch.tensor([v - 1, 0, v // 2], dtype=torch.int32, device=DEV)
    big = torch.empty(n, ld, device=DEV, dtype=torch.bfloat16)
    big[:, :d], big[:, 64:64 + d] = s["x"], s["w"]
    t = {**s, "x": big[:, :d], "w": big[:, 64:64 + d]}
    handle = mt.CrossEntropy(v, d)
    r = handle.forward(t["x"], t["w"], t["targets"])
    dx, dw = handle.backward(t["dloss"], t["x"], t["w"], t["targets"], r.lse, out_dx=big[:, 128:128 + d])
    # the rows that take part, against the definition (the sums' runs go by n, so another n need not give the same bits)
    live = s["targets"] >= 0
    assert not r.loss[~live].any() and not r.lse[~live].any() and not dx[~live].any()
    c = {**s, "x": s["x"][live], "targets": s["targets"][live], "dloss": s["dloss"][live]}
    check_all(c, "bf16", handle=handle, forward=mt.LossForward(r.loss[live], r.lse[live]), grads=(dx[live], dw))


def test_gradients_against_differences():
    """fp32, along random directions; differences of the library's own losses."""
    for top in (0, 5):
        s = make(14, 40, 90, 24, "f32", top=top)
        handle = mt.CrossEntropy(90, 24, smoothing=0.1, z_loss=1e-2, dtype="f32") if top == 0 else mt.Distillation(90, 24, top, dtype="f32")
        r = handle.forward(s["x"], s["w"], *given(s))
        grads = handle.backward(s["dloss"], s["x"], s["w"], *given(s), r.lse)
        gen = torch.Generator(device=DEV).manual_seed(15)
        for what, grad in zip(("x", "w"), grads):
            v = torch.randn(grad.shape, generator=gen, device=DEV)
            out, step = [], 2.0 ** -7
            for h in (step, -step):
                t = {**s, what: s[what] + h * v}
                out.append((s["dloss"].double() * handle.forward(t["x"], t["w"], *given(t)).loss.double()).sum())
            diff = (out[0] - out[1]) / (2 * step)
            size = float((grad.double() * v.double()).abs().sum())
            assert abs(float(diff) - float((grad.double() * v.double()).sum())) <= 2e-3 * size, (top, what)


def test_refusals():
    s = make(16, 30, 50, 64, "bf16")
    handle = mt.CrossEntropy(50, 64)
    for bad in (dict(vocab=0), dict(dim=0), dict(dim=8193), dict(vocab=2 ** 31 - 4095), dict(scale=0.0), dict(scale=float("nan")), dict(smoothing=1.0),
                dict(smoothing=-0.1), dict(z_loss=-1.0)):
        with pytest.raises(mt.MTError):
            mt.CrossEntropy(**{**dict(vocab=50, dim=64), **bad})
    for top in (0, 1025):
        with pytest.raises(mt.MTError):
            mt.Distillation(50, 64, top)
    with pytest.raises(TypeError):
        handle.forward(s["x"].float(), s["w"], s["targets"])
    with pytest.raises(TypeError):
        handle.forward(s["x"], s["w"], s["targets"].short())
    with pytest.raises(ValueError):
        handle.forward(s["x"], s["w"][:-1], s["targets"])
    with pytest.raises(ValueError):
        handle.forward(s["x"], s["w"], s["targets"][:-1])
    with pytest.raises(ValueError):
        handle.forward(s["x"], s["w"], torch.stack([s["targets"]] * 2, 1)[:, 0])  # not contiguous
    r = handle.forward(s["x"], s["w"], s["targets"])
    with pytest.raises(ValueError):
        handle.backward(s["dloss"].double(), s["x"], s["w"], s["targets"], r.lse)
    with pytest.raises(ValueError):
        handle.backward(s["dloss"], s["x"], s["w"], s["targets"], r.lse, want_dx=False, want_dw=False)
    with pytest.raises(mt.MTError):
        handle.backward(s["dloss"], s["x"], s["w"], s["targets"], r.lse, out_dx=s["x"])
    with pytest.raises(mt.MTError):
        handle.backward(s["dloss"], s["x"], s["w"], s["targets"], r.lse, out_dw=s["w"])
    d = mt.Distillation(50, 64, 3)
    with pytest.raises(TypeError):
        d.forward(s["x"], s["w"], torch.zeros(30, 3, dtype=torch.int32, device=DEV), torch.zeros(30, 3, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError):
        d.forward(s["x"], s["w"], torch.zeros(30, 3, dtype=torch.int32, device=DEV), torch.zeros(30, 2, device=DEV))

"""The losses over a vocabulary where a call's shape or values leave the common path; tolerances as in test_gpu_loss."""
import math

import pytest
import torch

import update_merged_table_gb300 as mt
from test_gpu_loss import DEV, check_all, given, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,v,d,top", [(100, 30000, 64, 0), (65, 40001, 16, 0), (128, 30000, 64, 3), (30000, 100, 64, 0), (25000, 128, 40, 0)])
def test_sums_of_one_tile(n, v, d, top):
    """Narrow rows whose gradients' sums have one tile of logits each and several to a block: teams without a tile in a sum."""
    s = make(41, n, v, d, "bf16", top=top, masked=0.0)
    handle, r, (dx, dw) = check_all(s, "bf16")
    for _ in range(30):
        ax, aw = handle.backward(s["dloss"], s["x"], s["w"], *given(s), r.lse)
        assert torch.equal(ax, dx) and torch.equal(aw, dw)
    assert handle.error() == 0


@pytest.mark.parametrize("n,v,d", [(100, 700, 200), (2048, 20000, 256), (4096, 5000, 512), (2048, 20000, 640), (300, 2500, 1032)])
@pytest.mark.parametrize("scale,smoothing,z_loss", [(1.5, 0.3, 1e-3), (0.5, 0.1, 0.0)])
def test_smoothing_and_z_loss_of_wide_rows(n, v, d, scale, smoothing, z_loss):
    """Tiles of 256 entries, by blocks and by pairs, whose rows of x stay with the block and whose do not."""
    check_all(make(42, n, v, d, "bf16"), "bf16", scale, smoothing, z_loss)


@pytest.mark.parametrize("n,v,d,top", [(2048, 20000, 256, 16), (2048, 20000, 640, 5), (100, 700, 200, 8)])
def test_scale_of_distillation_over_wide_rows(n, v, d, top):
    check_all(make(43, n, v, d, "bf16", top=top), "bf16", scale=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kept", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [0.5, 2.0, 3.0])
def test_teachers_of_the_largest_and_lowest_logits(scale, kept, dtype):
    """A kept logit of the type's lowest value (a mask of the teacher's) is a pair like others: equal ones share, and beside any
    other it has nothing; times the scale it is no fp32 number."""
    low = torch.finfo(kept).min
    s = make(44, 6, 50, 32, dtype, top=4, masked=0.0)
    s["ids"] = torch.tensor([[3, 9, 4, 7], [1, 2, 0, 4], [9, 9, 8, 7], [5, 6, -1, -1], [8, 0, 49, 8], [-1, 6, 6, -1]], dtype=torch.int32, device=DEV)
    s["logits"] = torch.tensor([[low, low, low, low], [1.0, low, 2.0, low], [-low, low, 0.0, -low], [-low, -low, low, 0.0],
                                [low, low / 2, low, low], [0.0, low, low, -low]], device=DEV).to(kept)
    _, r, (dx, dw) = check_all(s, dtype, scale=scale)
    assert bool(torch.isfinite(r.loss).all()) and bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("n,top", [(2, 1024), (300, 1024), (40, 1023), (3, 513), (70, 129), (70, 128), (70, 127), (70, 65), (70, 64), (70, 63), (9, 33)])
def test_long_lists_of_a_teacher(n, top):
    """Lists sorted in every way there is; many of the same id, and ids in descending order."""
    s = make(47, n, 200, 24, "f32", top=top, masked=0.1)
    s["ids"][0] = torch.arange(top, 0, -1, device=DEV, dtype=torch.int32) % 200
    s["ids"][-1] = 7
    check_all(s, "f32")


@pytest.mark.parametrize("n,top", [(2, 1024), (1, 1024), (16, 128), (15, 130), (64, 32), (33, 62), (255, 8), (256, 8), (257, 8), (1024, 2), (1025, 2)])
def test_rows_marked_by_their_pairs(n, top):
    """Up to 2048 pairs a block looks through all of them; rows whose only pair comes last, rows without any, and pairs outside
    the vocabulary in rows that take part and in rows that do not."""
    v, d = 700, 24
    s = make(45, n, v, d, "f32", top=top, masked=0.0)
    for i in range(0, n, 3):
        s["ids"][i] = -1
        if i % 2 == 0:
            s["ids"][i, -1] = i % v
    check_all(s, "f32")
    handle = mt.Distillation(v, d, top, dtype="f32")
    bad = s["ids"].clone()
    bad[0], bad[-1, -1] = v, 2 ** 31 - 1
    safe = torch.where(bad >= v, -1, bad)
    r = handle.forward(s["x"], s["w"], bad, s["logits"])
    assert handle.error(clear=True) == mt.MT_EINVAL
    want = handle.forward(s["x"], s["w"], safe, s["logits"])
    assert torch.equal(r.loss, want.loss) and torch.equal(r.lse, want.lse) and float(r.loss[0]) == 0 and handle.error() == 0


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2047, 2048, 2049])
def test_rows_marked_by_their_targets(n):
    check_all(make(46, n, 300, 24, "bf16", masked=0.5), "bf16")


@pytest.mark.parametrize("n,v,d", [(152 * 128, 1 << 21, 16), (1 << 21, 152 * 128 + 5, 16), (152 * 128, 1 << 20, 128), (2176, 900_000, 2056),
                                   (640, 2_700_000, 8192), (900_000, 2304, 2056), (1_500_000, 1024, 4096)])
def test_sums_of_many_equal_terms(n, v, d):
    """Over a million terms of one sign and size, whose every addition the tensor core cuts off: at most 2^-23 of the sum for 16
    of them, so at most 2^-9 in the 2^18 after which a sum starts anew at the latest; then the gradient's own rounding."""
    t, w0 = v // 3, 2.0 ** -math.ceil(math.log2(d))
    x, w = torch.ones(n, d, device=DEV, dtype=torch.bfloat16), torch.full((v, d), w0, device=DEV, dtype=torch.bfloat16)
    w[t] = 0.0
    targets = torch.full((n,), t, device=DEV, dtype=torch.int32)
    z = d * w0
    lse = math.log((v - 1) * math.exp(z) + 1.0)
    dz = 255.0 * 2.0 ** -30  # as bf16 has it
    handle = mt.CrossEntropy(v, d)
    dx, dw = handle.backward(torch.full((n,), dz / math.exp(z - lse), device=DEV), x, w, targets, torch.full((n,), lse, device=DEV))
    tol = 2.0 ** -8 + 2.0 ** -9 + 1e-5
    keep = torch.arange(v, device=DEV) != t
    for got, want in ((dx, (v - 1) * dz * w0), (dw[keep], n * dz)):
        least, most = float(got.min()) / want, float(got.max()) / want
        assert 1.0 - tol <= least <= most <= 1.0 + tol
    assert handle.error() == 0


@pytest.mark.parametrize("n,v,d", [(64, 5000, 40), (65, 5000, 40), (65, 5000, 256), (2000, 3000, 64), (2000, 3000, 256)])
def test_padded_batches(n, v, d):
    """Two rows that take part among many that do not: the gradient of their logits is rounded by what all rows are, and the
    results stay within what that rounding allows."""
    s = make(48, n, v, d, "bf16", masked=0.0)
    keep = torch.zeros(n, dtype=torch.bool, device=DEV)
    keep[[n // 3, n - 1]] = True
    s["targets"][~keep] = -1
    s["dloss"] = torch.full((n,), 0.5, device=DEV)
    _, _, (dx, dw) = check_all(s, "bf16")
    # without the padding: the same within both sides' rounding of the logits' gradient and of the result, 2^-8 each
    few = {k: (t if k == "w" else t[keep]).contiguous() for k, t in s.items()}
    _, _, (dx2, dw2) = check_all(few, "bf16")
    for a, b in ((dx[keep], dx2), (dw, dw2)):
        assert float((a.double() - b.double()).norm()) <= 4 * 2.0 ** -8 * float(b.double().norm())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,d,top", [(130, 600, 8192, 0), (300, 520, 8191, 3), (3, 1, 8192, 0), (5000, 1, 64, 0), (5000, 2, 1, 2), (40, 1, 24, 1024),
                                       (1, 2, 8192, 1024), (1, 70001, 1, 0), (700_001, 3, 8, 0), (300_001, 50, 136, 0)])
def test_smallest_and_largest_sizes(n, v, d, top, dtype):
    check_all(make(49, n, v, d, dtype, top=top), dtype, scale=0.5 if top else 1.0)


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 50.0])
def test_small_and_large_scales(scale):
    for dtype in ("bf16", "f32"):
        check_all(make(50, 200, 300, 72, dtype), dtype, scale=scale, smoothing=0.1)
        check_all(make(51, 200, 300, 72, dtype, top=5), dtype, scale=scale)


def test_captured_calls_behind_a_join():
    """Kernels that follow others by programmatic launches, captured right behind events of other streams, copies and fills."""
    s = make(52, 600, 4000, 200, "bf16")
    t = make(53, 300, 2000, 64, "bf16", top=7)
    ce, kd = mt.CrossEntropy(4000, 200), mt.Distillation(2000, 64, 7)
    ffn = mt.GatedLinear(2, 200, 64)
    gen = torch.Generator(device=DEV).manual_seed(54)
    w1 = (torch.randn(2, 128, 200, generator=gen, device=DEV) * 0.1).bfloat16()
    off = torch.tensor([0, 100, 600], device=DEV)
    x, x2 = s["x"].clone(), t["x"].clone()

    def step(side):
        main = torch.cuda.current_stream()
        x.copy_(s["x"])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x2.copy_(t["x"])
            k = kd.forward(x2, t["w"], t["ids"], t["logits"])
            gk = kd.backward(t["dloss"], x2, t["w"], t["ids"], t["logits"], k.lse)
        r = ce.forward(x, s["w"], s["targets"])
        gr = ce.backward(s["dloss"], x, s["w"], s["targets"], r.lse)
        main.wait_stream(side)
        h = ffn.forward(gr[0], w1, off)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            back = ffn.backward(h, gr[0], w1, off)
        main.wait_stream(side)
        return (r.loss, *gr, k.loss, *gk, h, *back)

    side = torch.cuda.Stream()
    want = [a.clone() for a in step(side)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(torch.cuda.Stream())
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for a in got:
            a.zero_()
    assert not ce.error() and not kd.error() and not ffn.error()

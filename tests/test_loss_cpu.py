"""The gated feed-forward part and the losses without a GPU: the C calls refuse bad arguments on the host before any device
call, and the 64-bit reference that the GPU tests compare with is checked against differences."""
import ctypes

import pytest
import torch

import loss_reference as R
import update_merged_table_gb300 as mt
from test_block_cpu import P, lib  # noqa: F401 (lib: the built library)

MOST = (1 << 31) - 4096


class Gated(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("in_dim", ctypes.c_int32), ("out_dim", ctypes.c_int32), ("groups", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("reserved", ctypes.c_int32), ("offsets", ctypes.c_void_p), ("status", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("w", ctypes.c_void_p)]


class Vocab(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("vocab", ctypes.c_int32), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("top", ctypes.c_int32),
                ("scale", ctypes.c_float), ("smoothing", ctypes.c_float), ("z_loss", ctypes.c_float), ("id_bytes", ctypes.c_int32),
                ("teacher_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("w", ctypes.c_void_p),
                ("ldw", ctypes.c_int64), ("targets", ctypes.c_void_p), ("teacher", ctypes.c_void_p), ("status", ctypes.c_void_p)]


def gated(**kw):
    base = {**dict(n=8, in_dim=64, out_dim=32, groups=2, dtype=mt.MT_BF16, gate=3, reserved=0, offsets=P, status=None, x=2 * P, ldx=64, w=3 * P), **kw}
    return Gated(*[base[f] for f, _ in Gated._fields_])


def vocab(**kw):
    base = {**dict(n=8, vocab=50, dim=64, dtype=mt.MT_BF16, top=0, scale=1.0, smoothing=0.0, z_loss=0.0, id_bytes=4, teacher_dtype=0, reserved=0, x=2 * P,
                   ldx=64, w=3 * P, ldw=64, targets=4 * P, teacher=None, status=None), **kw}
    return Vocab(*[base[f] for f, _ in Vocab._fields_])


def test_gated_refusals(lib):  # noqa: F811
    for bad in (dict(n=-1), dict(n=MOST + 1), dict(in_dim=0), dict(in_dim=8193), dict(out_dim=0), dict(out_dim=8193), dict(groups=0), dict(groups=1025),
                dict(dtype=2), dict(gate=0), dict(gate=5), dict(offsets=None), dict(offsets=P + 4), dict(status=P + 2), dict(x=None), dict(x=2 * P + 1),
                dict(ldx=63), dict(ldx=1 << 31), dict(w=None), dict(w=3 * P + 1)):
        c = gated(**bad)
        assert lib.mt_gated_linear_workspace_bytes(ctypes.byref(c), 1) == 0, bad
        assert lib.mt_gated_linear_forward(ctypes.byref(c), 5 * P, 32, 6 * P, 1 << 40, None) == mt.MT_EINVAL, bad
        assert lib.mt_gated_linear_backward(ctypes.byref(c), 5 * P, 32, 6 * P, 64, 7 * P, 8 * P, 1 << 40, None) == mt.MT_EINVAL, bad
    assert lib.mt_gated_linear_forward(None, P, 32, None, 0, None) == mt.MT_EINVAL
    c = gated()
    assert lib.mt_gated_linear_workspace_bytes(ctypes.byref(c), 0) == 0  # fits as it is
    odd = gated(in_dim=50)
    forward, backward = (lib.mt_gated_linear_workspace_bytes(ctypes.byref(odd), k) for k in (0, 1))
    assert 0 < forward < backward
    for h, ldh in ((None, 32), (5 * P + 1, 32), (5 * P, 31), (2 * P, 32)):  # the last: over x
        assert lib.mt_gated_linear_forward(ctypes.byref(c), h, ldh, None, 0, None) == mt.MT_EINVAL
    for ws, size in ((None, 1 << 30), (6 * P + 16, 1 << 30), (6 * P, forward - 1)):
        assert lib.mt_gated_linear_forward(ctypes.byref(odd), 5 * P, 32, ws, size, None) == mt.MT_ENOSPACE
    size = lib.mt_gated_linear_workspace_bytes(ctypes.byref(c), 1)

    def back(dh=5 * P, lddh=32, dx=6 * P, lddx=64, dw=7 * P, ws=8 * P, nb=size):
        return lib.mt_gated_linear_backward(ctypes.byref(c), dh, lddh, dx, lddx, dw, ws, nb, None)

    for kw in (dict(dh=None), dict(lddh=31), dict(dx=None, dw=None), dict(lddx=63), dict(dw=7 * P + 1), dict(dx=2 * P), dict(dw=3 * P), dict(dx=7 * P),
               dict(dx=5 * P), dict(ws=7 * P)):
        assert back(**kw) == mt.MT_EINVAL, kw
    for kw in (dict(ws=None), dict(ws=8 * P + 128), dict(nb=size - 1)):
        assert back(**kw) == mt.MT_ENOSPACE, kw
    assert lib.mt_gated_linear_forward(ctypes.byref(gated(n=0, x=None)), None, 0, None, 0, None) == mt.MT_OK


def test_loss_refusals(lib):  # noqa: F811
    for bad in (dict(n=-1), dict(n=MOST + 1), dict(vocab=0), dict(vocab=MOST + 1), dict(dim=0), dict(dim=8193), dict(dtype=2), dict(top=-1), dict(top=1025),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(smoothing=1.0), dict(smoothing=float("nan")),
                dict(z_loss=-1.0), dict(id_bytes=2), dict(top=2), dict(top=2, teacher=5 * P, smoothing=0.1), dict(top=2, teacher=5 * P, z_loss=0.1),
                dict(top=2, teacher=5 * P, teacher_dtype=2), dict(top=2, teacher=5 * P + 2), dict(x=None), dict(x=2 * P + 1), dict(ldx=63), dict(w=None),
                dict(ldw=63), dict(ldw=1 << 31), dict(targets=None), dict(targets=4 * P + 2), dict(targets=4 * P + 4, id_bytes=8), dict(status=P + 2)):
        c = vocab(**bad)
        assert lib.mt_vocab_loss_workspace_bytes(ctypes.byref(c), 0) == 0, bad
        assert lib.mt_vocab_loss_forward(ctypes.byref(c), 6 * P, 7 * P, 8 * P, 1 << 40, None) == mt.MT_EINVAL, bad
        assert lib.mt_vocab_loss_backward(ctypes.byref(c), 6 * P, 7 * P, 8 * P, 64, 9 * P, 10 * P, 1 << 40, None) == mt.MT_EINVAL, bad
    assert lib.mt_vocab_loss_forward(None, P, P, None, 0, None) == mt.MT_EINVAL
    c = vocab()
    size = lib.mt_vocab_loss_workspace_bytes(ctypes.byref(c), 0)
    far = 1 << 40

    def fore(loss=6 * P, lse=7 * P, ws=far, nb=size):
        return lib.mt_vocab_loss_forward(ctypes.byref(c), loss, lse, ws, nb, None)

    for kw in (dict(loss=None), dict(lse=None), dict(loss=6 * P + 2), dict(lse=6 * P), dict(loss=2 * P), dict(lse=4 * P), dict(loss=far)):
        assert fore(**kw) == mt.MT_EINVAL, kw
    for kw in (dict(ws=None), dict(ws=far + 16), dict(nb=size - 1)):
        assert fore(**kw) == mt.MT_ENOSPACE, kw
    size = lib.mt_vocab_loss_workspace_bytes(ctypes.byref(c), 1)

    def back(dloss=6 * P, lse=7 * P, dx=8 * P, lddx=64, dw=9 * P, ws=far, nb=size):
        return lib.mt_vocab_loss_backward(ctypes.byref(c), dloss, lse, dx, lddx, dw, ws, nb, None)

    for kw in (dict(dloss=None), dict(lse=None), dict(dx=None, dw=None), dict(lddx=63), dict(dw=9 * P + 1), dict(dx=2 * P), dict(dw=3 * P), dict(dx=9 * P),
               dict(dw=6 * P), dict(dx=far)):
        assert back(**kw) == mt.MT_EINVAL, kw
    for kw in (dict(ws=None), dict(ws=far + 128), dict(nb=size - 1)):
        assert back(**kw) == mt.MT_ENOSPACE, kw
    assert lib.mt_vocab_loss_forward(ctypes.byref(vocab(n=0, x=None, targets=None)), None, None, None, 0, None) == mt.MT_OK


@pytest.mark.parametrize("kind", ["linear", "sigmoid", "silu", "gelu"])
def test_gated_reference_against_differences(kind):
    gen = torch.Generator().manual_seed(1)
    x, w, dh = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((9, 6), (3, 10, 6), (9, 5)))
    off = torch.tensor([1, 4, 4, 8])
    r = R.gated(x, w, off, kind, dh)
    for what, grad in (("x", r["dx"]), ("w", r["dw"])):
        v = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
        out = []
        for s in (1e-5, -1e-5):
            h = R.gated(x + s * v if what == "x" else x, w + s * v if what == "w" else w, off, kind)["h"]
            out.append(float((dh * h).sum()))
        assert abs((out[0] - out[1]) / 2e-5 - float((grad * v).sum())) <= 1e-7 * (float((grad * v).abs().sum()) + 1.0)


@pytest.mark.parametrize("distill", [False, True])
def test_loss_reference_against_differences(distill):
    gen = torch.Generator().manual_seed(2)
    x, w, g = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((9, 6), (11, 6), (9,)))
    if distill:
        ids = torch.randint(-2, 11, (9, 4), generator=gen)
        ids[3] = -1
        more = dict(ids=ids, logits=torch.randn(9, 4, generator=gen, dtype=torch.float64))
    else:
        more = dict(targets=torch.randint(-1, 11, (9,), generator=gen), smoothing=0.2, z_loss=0.05)
    r = R.loss(x, w, 0.7, dloss=g, **more)
    for what, grad in (("x", r["dx"]), ("w", r["dw"])):
        v = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
        out = [float((g * R.loss(x + s * v if what == "x" else x, w + s * v if what == "w" else w, 0.7, **more)["loss"]).sum()) for s in (1e-5, -1e-5)]
        assert abs((out[0] - out[1]) / 2e-5 - float((grad * v).sum())) <= 1e-7 * (float((grad * v).abs().sum()) + 1.0)


def test_cross_entropy_reference_is_the_mean_of_log_probabilities():
    gen = torch.Generator().manual_seed(3)
    x, w = torch.randn(5, 4, generator=gen, dtype=torch.float64), torch.randn(7, 4, generator=gen, dtype=torch.float64)
    t = torch.tensor([0, 6, 3, 3, 1])
    want = torch.nn.functional.cross_entropy(x @ w.T, t, label_smoothing=0.1, reduction="none")
    assert torch.allclose(R.loss(x, w, targets=t, smoothing=0.1)["loss"], want, rtol=1e-12)

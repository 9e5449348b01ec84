"""The dense block without a GPU: the C calls refuse bad arguments on the host before any device call, and the 64-bit
reference that the GPU tests compare with is checked against differences and against its own definition."""
import ctypes

import numpy as np
import pytest

import block_reference as R
import update_merged_table_gb300 as mt
from update_merged_table_gb300 import build_lib


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("codes", ctypes.c_void_p), ("exps", ctypes.c_void_p)]


class Norm(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("dim", ctypes.c_int32), ("groups", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("kind", ctypes.c_int32), ("gate", ctypes.c_int32), ("eps", ctypes.c_float), ("offsets", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p), ("pre_bias", ctypes.c_void_p)]


P = 1 << 20  # a stand-in address: nothing is read or launched


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return mt.load_library()


def test_pack_refusals(lib):
    for bad in (dict(x=None), dict(x=P + 1), dict(ldx=63), dict(n=-1), dict(n=1 << 31), dict(d=0), dict(d=8193), dict(dtype=2),
                dict(codes=None), dict(exps=None), dict(ldx=1 << 31)):
        a = {**dict(x=P, ldx=64, n=4, d=64, dtype=mt.MT_BF16, codes=P, exps=P), **bad}
        assert lib.mt_pack8(a["x"], a["ldx"], a["n"], a["d"], a["dtype"], a["codes"], a["exps"], None) == mt.MT_EINVAL, bad
        assert lib.mt_unpack8(a["codes"], a["exps"], a["n"], a["d"], a["dtype"], a["x"], a["ldx"], None) == mt.MT_EINVAL, bad
    assert lib.mt_pack8(None, 64, 0, 64, mt.MT_F32, None, None, None) == mt.MT_OK  # no rows: nothing to do


def test_linear_refusals(lib):
    base = dict(x=P, ldx=64, w=P, off=P, g=2, n=8, k=64, m=32, dtype=mt.MT_BF16, y=P, ldy=32, status=None)
    for bad in (dict(x=None), dict(x=P + 1), dict(ldx=63), dict(w=None), dict(off=None), dict(off=P + 4), dict(g=0), dict(g=1025),
                dict(n=-1), dict(n=1 << 31), dict(k=0), dict(k=8193), dict(m=0), dict(m=9000), dict(dtype=5), dict(y=None),
                dict(ldy=31), dict(status=P + 2)):
        a = {**base, **bad}
        assert lib.mt_group_linear_forward(a["x"], a["ldx"], a["w"], a["off"], a["g"], a["n"], a["k"], a["m"], a["dtype"], a["y"],
                                           a["ldy"], a["status"], None) == mt.MT_EINVAL, bad
    ws = lib.mt_group_linear_workspace_bytes(8, 2, 64, 32)
    assert ws > 0
    for args in ((-1, 2, 64, 32), (8, 0, 64, 32), (8, 1025, 64, 32), (8, 2, 0, 32), (8, 2, 64, 9000)):
        assert lib.mt_group_linear_workspace_bytes(*args) == 0
    x = Rows(P, 64, None, None)
    base = dict(dy=P, lddy=32, x=ctypes.byref(x), w=P, off=P, g=2, n=8, k=64, m=32, dtype=mt.MT_BF16, dx=P, lddx=64, dw=P,
                ws=P, nb=ws)
    for bad, code in ((dict(dy=None), mt.MT_EINVAL), (dict(lddy=31), mt.MT_EINVAL), (dict(x=None), mt.MT_EINVAL),
                      (dict(x=ctypes.byref(Rows())), mt.MT_EINVAL), (dict(x=ctypes.byref(Rows(None, 0, P, None))), mt.MT_EINVAL),
                      (dict(w=None), mt.MT_EINVAL), (dict(dx=None, dw=None), mt.MT_EINVAL), (dict(lddx=63), mt.MT_EINVAL),
                      (dict(dw=P + 2), mt.MT_EINVAL), (dict(ws=None), mt.MT_ENOSPACE), (dict(ws=P + 16), mt.MT_ENOSPACE),
                      (dict(nb=ws - 1), mt.MT_ENOSPACE), (dict(off=None), mt.MT_EINVAL)):
        a = {**base, **bad}
        assert lib.mt_group_linear_backward(a["dy"], a["lddy"], a["x"], a["w"], a["off"], a["g"], a["n"], a["k"], a["m"], a["dtype"],
                                            a["dx"], a["lddx"], a["dw"], None, a["ws"], a["nb"], None) == code, bad


def norm_config(**kw):
    base = dict(n=8, dim=64, groups=1, dtype=mt.MT_BF16, kind=0, gate=3, eps=1e-6, offsets=None, status=None, post_weight=P,
                post_bias=None, scale=P, pre_weight=P, pre_bias=None)
    base.update(kw)
    return Norm(*[base[f] for f, _ in Norm._fields_])


def test_norm_refusals(lib):
    row, none = Rows(P, 64, None, None), Rows()
    half = Rows(P, 64, P, None)

    def forward(c=None, x=row, y=row, u=row, z=row, h=row):
        return lib.mt_gated_norm_forward(ctypes.byref(c if c is not None else norm_config()), *(ctypes.byref(r) for r in (x, y, u, z, h)), None)

    for kw in (dict(n=-1), dict(dim=0), dict(dim=8193), dict(groups=0), dict(groups=1025), dict(groups=2), dict(dtype=3), dict(kind=2),
               dict(gate=4), dict(eps=0.0), dict(eps=float("nan")), dict(offsets=P + 4), dict(status=P + 1), dict(post_weight=None),
               dict(gate=0), dict(post_weight=P + 2), dict(pre_weight=None)):
        assert forward(norm_config(**kw)) == mt.MT_EINVAL, kw
    for kw in (dict(x=none), dict(x=half), dict(y=none), dict(u=none), dict(z=none), dict(h=none), dict(y=half), dict(z=half), dict(x=Rows(P, 63)),
               dict(h=Rows(P + 1, 64)), dict(y=Rows(P, 1 << 31))):
        assert forward(**kw) == mt.MT_EINVAL, kw
    assert lib.mt_gated_norm_forward(None, None, None, None, None, None, None) == mt.MT_EINVAL
    ws = lib.mt_gated_norm_workspace_bytes(8, 64, 1)
    assert ws > 0 and lib.mt_gated_norm_workspace_bytes(-1, 64, 1) == 0 and lib.mt_gated_norm_workspace_bytes(8, 0, 1) == 0
    assert lib.mt_gated_norm_workspace_bytes(8, 64, 1025) == 0
    packed = Rows(None, 0, P, P)

    def backward(c=None, nb=ws, w=P, grads=(P, None, P, P, None), **kw):
        r = {**dict(dz=row, dh=row, y=packed, u=row, z=packed, dx=row, dy=row, du=row), **kw}
        return lib.mt_gated_norm_backward(ctypes.byref(c if c is not None else norm_config()),
                                          *(ctypes.byref(r[k]) for k in ("dz", "dh", "y", "u", "z", "dx", "dy", "du")), *grads, w, nb, None)

    for kw in (dict(dh=none), dict(y=none), dict(u=none), dict(z=none), dict(dx=none), dict(dy=none), dict(du=none), dict(dz=packed),
               dict(dx=packed), dict(z=half if half.data is None else Rows(None, 0, P, None)), dict(grads=(None, None, P, P, None)),
               dict(grads=(P, P, P, P, None)), dict(grads=(P, None, P, P + 1, None)), dict(dz=Rows(P, 60))):
        assert backward(**kw) == mt.MT_EINVAL, kw
    assert backward(w=None) == mt.MT_ENOSPACE and backward(nb=ws - 1) == mt.MT_ENOSPACE and backward(w=P + 128) == mt.MT_ENOSPACE


def test_reference_pack_is_the_least_exponent():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 70)) * np.exp(10 * rng.standard_normal((50, 1)))).astype(np.float32)
    x[3], x[4, :32] = 0.0, 127.0
    codes, exps = R.pack(x)
    back = R.unpack(codes, exps)
    e = exps.astype(int) - 127
    for b in range(3):
        top = np.abs(x[:, 32 * b:32 * b + 32]).max(1).astype(np.float64)
        live = top > 0
        assert (top <= np.ldexp(127.0, e[:, b]))[live].all()
        assert ((top > np.ldexp(127.0, e[:, b] - 1)) | (e[:, b] == -120))[live].all()
        assert (np.abs(back - x)[:, 32 * b:32 * b + 32] <= np.ldexp(0.5, e[:, b])[:, None]).all()
    import torch
    t = torch.from_numpy(back)
    assert torch.equal(t.to(torch.bfloat16).double(), t)  # every value is a bf16 number


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "linear", "sigmoid", "silu"])
def test_reference_gradients_against_differences(kind, gate):
    rng = np.random.default_rng(1)
    n, d, off = 7, 12, np.array([1, 4, 4, 6])
    p = {k: 1.0 + 0.3 * rng.standard_normal((3, d)) for k in ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")}
    a = {k: rng.standard_normal((n, d)) for k in ("x", "y", "u")}
    if gate == "none":
        a["u"] = None
    dz, dh = rng.standard_normal((n, d)), rng.standard_normal((n, d))
    z, _ = R.norm_forward(a["x"], a["y"], a["u"], p, off, kind, gate, 1e-5)
    got, _ = R.norm_backward(dz, dh, a["y"], a["u"], z, p, off, kind, gate, 1e-5)
    got = {"x": got["dx"], "y": got["dy"], **({"u": got["du"]} if gate != "none" else {}), **{k: got[k] for k in p}}

    def loss(values, params):
        zz, hh = R.norm_forward(values["x"], values["y"], values["u"], params, off, kind, gate, 1e-5)
        return (dz * zz).sum() + (dh * hh).sum()

    for name, grad in got.items():
        v = rng.standard_normal(grad.shape)
        out = []
        for s in (1e-5, -1e-5):
            values = {k: t if k != name else t + s * v for k, t in a.items()}
            out.append(loss(values, {k: t if k != name else t + s * v for k, t in p.items()}))
        assert abs((out[0] - out[1]) / 2e-5 - (grad * v).sum()) <= 1e-7 * (np.abs(grad * v).sum() + 1.0), name

"""The dense block's operators in 64 bits on the CPU (numpy), from their formulas; no code shared with the library.

Every function takes float64 arrays holding the values the kernels were given.  ``norm_backward`` also returns, beside
each gradient, the size of what was added up to make it (sums of absolute values, also inside the terms: a term that is
small because its parts cancel keeps the rounding of its parts), which scales the tests' tolerances.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def spans(offsets):
    return [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def safe_offsets(offsets, n):
    """What bad offsets count as: clamped to [0, n], raised to their running maximum."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, n))


# ---- 8-bit checkpoints -----------------------------------------------------------------------------------------------

def pack(x):
    """(codes, exps) of float rows x, block by block."""
    n, d = x.shape
    nb = -(-d // BLOCK)
    codes = np.zeros((n, d), np.int8)
    exps = np.zeros((n, nb), np.uint8)
    for b in range(nb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
        top = np.abs(v).max(1)
        bad = ~np.isfinite(top)
        e = np.full(n, -120, np.int64)
        ok = ~bad & (top > 0)
        e[ok] = np.ceil(np.log2(top[ok] / 127.0) - 1e-9).astype(np.int64)  # a guess, then exact comparisons
        for _ in range(3):
            e = np.where(ok & (top > np.ldexp(127.0, e)), e + 1, e)
            e = np.where(ok & (top <= np.ldexp(127.0, e - 1)), e - 1, e)
        e = np.clip(e, -120, 121)
        with np.errstate(invalid="ignore"):
            q = np.clip(np.rint(np.ldexp(np.where(bad[:, None], 0.0, v), -e[:, None])), -127, 127)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = q.astype(np.int8)
        exps[:, b] = np.where(bad, 255, e + 127)
    return codes, exps


def unpack(codes, exps):
    e = exps.astype(np.int64)
    scale = np.where(e == 255, np.nan, np.ldexp(1.0, e - 127))
    return codes.astype(np.float64) * np.repeat(scale, BLOCK, axis=1)[:, :codes.shape[1]]


# ---- grouped products ------------------------------------------------------------------------------------------------

def linear_forward(x, w, offsets):
    """(y, sum of |products|)."""
    y = np.zeros((x.shape[0], w.shape[1]))
    size = np.zeros_like(y)
    for g, (a, b) in enumerate(spans(offsets)):
        y[a:b] = x[a:b] @ w[g].T
        size[a:b] = np.abs(x[a:b]) @ np.abs(w[g]).T
    return y, size


def linear_backward(dy, x, w, offsets):
    """(dx, its size, dw, its size)."""
    dx, sdx = np.zeros_like(x), np.zeros_like(x)
    dw, sdw = np.zeros(w.shape), np.zeros(w.shape)
    for g, (a, b) in enumerate(spans(offsets)):
        dx[a:b] = dy[a:b] @ w[g]
        sdx[a:b] = np.abs(dy[a:b]) @ np.abs(w[g])
        dw[g] = dy[a:b].T @ x[a:b]
        sdw[g] = np.abs(dy[a:b]).T @ np.abs(x[a:b])
    return dx, sdx, dw, sdw


# ---- gated norm -------------------------------------------------------------------------------------------------------

def _normed(v, kind, eps):
    if kind == "layer":
        v = v - v.mean(1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return v * r, r


def _norm_grad(g, vh, r, kind):
    out = g - vh * (g * vh).mean(1, keepdims=True)
    if kind == "layer":
        out = out - g.mean(1, keepdims=True)
    return out * r


def _gate(u, gate):
    if u is None:
        return 1.0, 0.0
    if gate == "linear":
        return u, np.ones_like(u)
    s = 1.0 / (1.0 + np.exp(-u))
    return (s, s * (1 - s)) if gate == "sigmoid" else (u * s, s * (1 + u * (1 - s)))


def _param(p, k, g, default):
    return p[k][g][None, :] if p.get(k) is not None else default


def norm_forward(x, y, u, p, offsets, kind, gate, eps):
    """(z, h or None); p: dict of float64 [groups, dim] or None."""
    z = np.zeros_like(x)
    h = np.zeros_like(x) if p.get("pre_weight") is not None else None
    for g, (a, b) in enumerate(spans(offsets)):
        z[a:b] = x[a:b]
        if y is not None:
            yh, _ = _normed(y[a:b], kind, eps)
            act, _ = _gate(u[a:b] if u is not None else None, gate)
            z[a:b] += _param(p, "scale", g, 1.0) * (_param(p, "post_weight", g, 1.0) * yh + _param(p, "post_bias", g, 0.0)) * act
        if h is not None:
            h[a:b] = _param(p, "pre_weight", g, 1.0) * _normed(z[a:b], kind, eps)[0] + _param(p, "pre_bias", g, 0.0)
    return z, h


def norm_backward(dz, dh, y, u, z, p, offsets, kind, gate, eps):
    """Gradients {dx, dy, du, post_weight, ...} and, for the parameters, {name: sum of |terms|}."""
    lead = dz if dz is not None else dh
    out = {"dx": np.zeros_like(lead)}
    if y is not None:
        out["dy"] = np.zeros_like(lead)
    if u is not None:
        out["du"] = np.zeros_like(lead)
    size = {}
    for k, v in p.items():
        if v is not None:
            out[k], size[k] = np.zeros_like(v), np.zeros_like(v)

    def add(k, g, terms, parts):
        if p.get(k) is not None:
            out[k][g], size[k][g] = terms.sum(0), parts.sum(0)

    def parts_of(v, r):  # |v| normalised, before the mean is taken off
        return (np.abs(v) + (np.abs(v.mean(1, keepdims=True)) if kind == "layer" else 0.0)) * r

    for g, (a, b) in enumerate(spans(offsets)):
        D = dz[a:b].copy() if dz is not None else np.zeros_like(lead[a:b])
        sD = np.abs(D)
        if dh is not None:
            zh, r = _normed(z[a:b], kind, eps)
            dzh, zp = dh[a:b] * _param(p, "pre_weight", g, 1.0), parts_of(z[a:b], r)
            D += _norm_grad(dzh, zh, r, kind)
            sD = sD + r * (np.abs(dzh) + np.abs(dzh).mean(1, keepdims=True) + zp * np.abs(dzh * zh).mean(1, keepdims=True))
            add("pre_weight", g, dh[a:b] * zh, np.abs(dh[a:b]) * zp)
            add("pre_bias", g, dh[a:b], np.abs(dh[a:b]))
        out["dx"][a:b] = D
        if y is not None:
            yh, r = _normed(y[a:b], kind, eps)
            act, dact = _gate(u[a:b] if u is not None else None, gate)
            w, s = _param(p, "post_weight", g, 1.0), _param(p, "scale", g, 1.0)
            t = w * yh + _param(p, "post_bias", g, 0.0)
            dt = D * s * act
            out["dy"][a:b] = _norm_grad(dt * w, yh, r, kind)
            if u is not None:
                out["du"][a:b] = D * s * t * dact
            yp, sdt = parts_of(y[a:b], r), sD * np.abs(s * act)
            add("post_weight", g, dt * yh, sdt * yp)
            add("post_bias", g, dt, sdt)
            add("scale", g, D * t * act, sD * np.abs(act) * (np.abs(w) * yp + np.abs(_param(p, "post_bias", g, 0.0))))
    return out, size

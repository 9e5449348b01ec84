"""The gated feed-forward part and the losses over a vocabulary in 64 bits (torch, on any device), from their formulas; no
code shared with the library.  Beside each result comes the size of what was added up to make it, which scales the tests'
tolerances."""
from __future__ import annotations

import math

import torch


def spans(offsets):
    o = offsets.tolist()
    return list(zip(o[:-1], o[1:]))


def gate(u, kind):
    """The gate's factor, its derivative, and a bound of the second derivative."""
    if kind == "linear":
        return u, torch.ones_like(u), 0.0
    if kind == "gelu":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(c * (u + 0.044715 * u ** 3))
        return u * s, s + u * s * (1 - s) * c * (1 + 3 * 0.044715 * u * u), 1.2
    s = torch.sigmoid(u)
    return (s, s * (1 - s), 0.1) if kind == "sigmoid" else (u * s, s * (1 + u * (1 - s)), 0.5)


def gated(x, w, offsets, kind, dh=None):
    """{y, u, sy, su, h} per row, and with dh {dy, du, dx, sdx, dw, sdw}: s... sums of absolute values."""
    n, m = x.shape[0], w.shape[1] // 2
    out = {k: torch.zeros(n, m, dtype=torch.float64, device=x.device) for k in ("y", "u", "sy", "su", "h", "dy", "du")}
    out["dx"], out["sdx"] = torch.zeros_like(x), torch.zeros_like(x)
    out["dw"], out["sdw"] = torch.zeros_like(w), torch.zeros_like(w)
    for g, (a, b) in enumerate(spans(offsets)):
        xg, wg = x[a:b], w[g]
        t, st = xg @ wg.T, xg.abs() @ wg.abs().T
        y, u = t[:, :m], t[:, m:]
        act, dact, _ = gate(u, kind)
        out["y"][a:b], out["u"][a:b], out["sy"][a:b], out["su"][a:b] = y, u, st[:, :m], st[:, m:]
        out["h"][a:b] = y * act
        if dh is not None:
            d = torch.cat([dh[a:b] * act, dh[a:b] * y * dact], 1)
            out["dy"][a:b], out["du"][a:b] = d[:, :m], d[:, m:]
            out["dx"][a:b], out["sdx"][a:b] = d @ wg, d.abs() @ wg.abs()
            out["dw"][g], out["sdw"][g] = d.T @ xg, d.abs().T @ xg.abs()
    return out


def shares(ids, logits, scale, vocab):
    """The teacher's distribution over a row's pairs, zero where a pair is not there; which rows have any."""
    there = (ids >= 0) & (ids < vocab) & (logits != -math.inf)
    s = torch.where(there, scale * logits, -math.inf)
    live = there.any(1)
    s = torch.where(live[:, None], s, 0.0)
    t = torch.where(there, torch.softmax(s, 1), 0.0)
    return t, torch.where(there, ids, 0).long(), live


def loss(x, w, scale=1.0, targets=None, smoothing=0.0, z_loss=0.0, ids=None, logits=None, dloss=None):
    """{loss, lse, live, p, z} and with dloss {dz, dx, dw, sdx, sdw}; everything of rows that take no part is zero."""
    v = w.shape[0]
    if targets is not None:
        live = (targets >= 0) & (targets < v)
        at = torch.where(live, targets, 0).long()[:, None]
        t = (1.0 - smoothing) * live.double()[:, None]
    else:
        t, at, live = shares(ids, logits, scale, v)
    x = torch.where(live[:, None], x, 0.0)
    z = scale * (x @ w.T)
    lse = torch.logsumexp(z, 1)
    out = {"live": live, "z": z, "sz": scale * (x.abs() @ w.abs().T)}
    value = lse + torch.xlogy(t, t).sum(1) * (targets is None) - (t * z.gather(1, at)).sum(1) - smoothing / v * z.sum(1) + z_loss * lse ** 2
    out["loss"], out["lse"] = torch.where(live, value, 0.0), torch.where(live, lse, 0.0)
    out["p"] = torch.exp(z - lse[:, None])
    if dloss is not None:
        g = torch.where(live, dloss, 0.0)[:, None]
        dz = out["p"] * (1.0 + 2.0 * z_loss * lse)[:, None] - smoothing / v
        dz.scatter_add_(1, at, -t)
        dz = dz * g * scale
        out["dz"] = dz
        out["dx"], out["dw"] = dz @ w, dz.T @ x
        out["sdx"], out["sdw"] = dz.abs() @ w.abs(), dz.abs().T @ x.abs()
    return out

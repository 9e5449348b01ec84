"""A small tower over a merged table: rows looked up, a gated block per layer, the gradient back into the table.

    python examples/dense_block.py --steps 50

A jagged batch's positions are grouped by feature (feature-major segments), and every part takes those groups as they
are: each feature has its own projection of the table's rows to the block's width, its own products and its own norm
parameters.  One layer is

    y | u = W h          one product makes the block's output and its gate side by side
    z     = x + s * norm(y) * silu(u)
    h'    = norm(z)      the next layer's input

Training keeps y, u, z and h in 8 bits (half of bf16) and the backward reads them there.  Weights are fp32, updated by
plain SGD, and cast to bf16 for the products.  ``Tower.serve`` is the same forward for single tokens, with nothing kept.

The targets are fixed random vectors, one per (feature, ID mod 97): something the table and the tower can learn.
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import update_merged_table_gb300 as mt  # noqa: E402
from update_merged_table_gb300 import workloads as W  # noqa: E402


@dataclasses.dataclass
class Kept:
    """What a layer's backward reads, in 8 bits."""
    h: mt.Packed8   # input of its product
    y: mt.Packed8
    u: mt.Packed8
    z: mt.Packed8   # residual stream after it

    @property
    def nbytes(self) -> int:
        return self.h.nbytes + self.y.nbytes + self.u.nbytes + self.z.nbytes


class Tower:
    def __init__(self, groups: int, row_dim: int, width: int, layers: int, device, seed: int = 0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(out, inp):
            return torch.randn(groups, out, inp, generator=gen, device=device) * inp ** -0.5

        def ones(scale=1.0):
            return torch.full((groups, width), scale, device=device)

        self.width = width
        self.embed = mt.GroupedLinear(groups, row_dim, width, device=device)
        self.linears = [mt.GroupedLinear(groups, width, 2 * width, device=device) for _ in range(layers)]
        self.first = mt.GatedNorm(width, num_groups=groups, kind="rms", gate="silu", device=device)
        self.norms = [mt.GatedNorm(width, num_groups=groups, kind="rms", gate="silu", device=device) for _ in range(layers)]
        self.w_embed = weight(width, row_dim)
        self.w = [weight(2 * width, width) for _ in range(layers)]
        self.p_first = mt.NormParams(pre_weight=ones())
        self.p = [mt.NormParams(post_weight=ones(), scale=ones(0.5), pre_weight=ones()) for _ in range(layers)]

    def forward(self, rows, offsets, keep: bool = True):
        """(h of the last layer, what the backward reads).  rows bf16 [n, row_dim], offsets int64 [groups + 1]."""
        x = self.embed.forward(rows, self.w_embed.bfloat16(), offsets)
        r = self.first.forward(x, params=self.p_first, offsets=offsets, pack="zh" if keep else "")
        first, kept = r.packed, []
        h8 = first.get("h")
        for lin, norm, w, p in zip(self.linears, self.norms, self.w, self.p):
            t = lin.forward(r.h, w.bfloat16(), offsets)
            d = self.width
            r = norm.forward(r.z, t[:, :d], t[:, d:], p, offsets, pack="yuzh" if keep else "")
            if keep:
                kept.append(Kept(h8, r.packed["y"], r.packed["u"], r.packed["z"]))
                h8 = r.packed["h"]
        return r.h, (rows, first, kept)

    def serve(self, rows, offsets):
        return self.forward(rows, offsets, keep=False)[0]

    def backward(self, dh, saved, offsets, lr: float):
        """The gradient of the table's rows; updates the weights and parameters on the way."""
        rows, first, kept = saved
        n, d = dh.shape
        dz = None
        for i in reversed(range(len(kept))):
            k, p = kept[i], self.p[i]
            dt = torch.empty((n, 2 * d), dtype=dh.dtype, device=dh.device)
            g = self.norms[i].backward(dz, dh, k.y, k.u, k.z, p, offsets, out_dy=dt[:, :d], out_du=dt[:, d:])
            dh, dw = self.linears[i].backward(dt, k.h, self.w[i].bfloat16(), offsets)
            dz = g.dx
            self.w[i].sub_(lr * dw)
            for name in ("post_weight", "scale", "pre_weight"):
                getattr(p, name).sub_(lr * getattr(g.params, name))
        g = self.first.backward(dz, dh, z=first["z"], params=self.p_first, offsets=offsets)
        drows, dw = self.embed.backward(g.dx, rows, self.w_embed.bfloat16(), offsets)
        self.w_embed.sub_(lr * dw)
        self.p_first.pre_weight.sub_(lr * g.params.pre_weight)
        return drows


def train(steps: int = 50, users: int = 64, features: int = 4, row_dim: int = 64, width: int = 128, layers: int = 2,
          log2_slots: int = 20, lr: float = 1.0, device=None, verbose: bool = True):
    """Runs the loop; returns the losses, one per step."""
    device = torch.device(device if device is not None else "cuda")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    table = mt.Table(log2_slots, row_dim, row_dtype="bf16", device=device)
    tower = Tower(features, row_dim, width, layers, device)
    goal = torch.randn(features, 97, width, generator=torch.Generator(device=device).manual_seed(1), device=device)
    losses = []
    for step in range(steps):
        b = W.jagged_batch(step, users=users, features=features)
        ids = torch.from_numpy(b.ids).to(device)
        offsets = torch.from_numpy(np.ascontiguousarray(b.feat_offsets, np.int64)).to(device)
        res = table.lookup(ids, b.feat_offsets, b.table_ids)
        h, saved = tower.forward(res.rows, offsets)
        feature = torch.searchsorted(offsets[1:], torch.arange(b.n, device=device), right=True)
        diff = h.float() - goal[feature, ids % 97]
        loss = 0.5 * diff.square().mean()
        dh = (diff / diff.numel()).bfloat16()
        drows = tower.backward(dh, saved, offsets, lr)
        table.backward_adam(res, drows, lr=1e-2)
        losses.append(float(loss))
        if verbose and (step % 10 == 0 or step + 1 == steps):
            kept = sum(k.nbytes for k in saved[2])
            print(f"step {step}: {b.n} positions, loss {losses[-1]:.4f}, kept {kept / 2 ** 20:.1f} MiB in 8 bits "
                  f"(bf16: {layers * 4 * b.n * width * 2 / 2 ** 20:.1f})")
    # serving: a token per feature, rows that the table has
    one = torch.arange(features, device=device)
    res = table.lookup(one, np.arange(features + 1), np.arange(features, dtype=np.uint8), insert_missing=False)
    h = tower.serve(res.rows, torch.arange(features + 1, device=device))
    assert h.shape == (features, width) and bool(torch.isfinite(h).all())
    errors = [table.error()] + [x.error() for x in (tower.embed, tower.first, *tower.linears, *tower.norms)]
    assert not any(errors), errors
    return losses


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--steps", type=int, default=50)
    a.add_argument("--users", type=int, default=64)
    a.add_argument("--width", type=int, default=128)
    a.add_argument("--layers", type=int, default=2)
    args = a.parse_args()
    train(args.steps, args.users, width=args.width, layers=args.layers)

"""The dense block between an embedding lookup and its gradient: the cases its operators are measured on.

Three operators over ragged groups of rows (a group is a feature segment of a jagged batch, or an expert's tokens):

* ``linear``: matrix products grouped by row segment, forward (y = x W_g^T) and backward (dx = dy W_g, dW_g = dy^T x).
* ``norm``: the norm after a block, its gate and its residual scale, the residual sum and the next block's norm in one
  pass, forward and backward.
* ``pack``: activation checkpoints in 8 bits (blocks of 32 columns with one power-of-two scale), written, read back, and
  read by the two backward passes.

Widths and row counts follow the repository's workloads: 16 to 128 columns per table row, 4096 to about two million IDs per
batch, about 490 thousand tokens of 2048 users; block widths of 256 to 2048 are generic.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 32        # columns that share a scale in a checkpoint
E_MIN, E_MAX = -120, 121
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token per request, eight requests, each with its own expert: latency and the experts' weights
        dict(name="linear 8 tokens", op="linear", way="fwd", dtype="bf16", n=8, groups=8, k=512, m=1024, skew=0.0),
        # the rows of a jagged batch's four features, each projected to the block's width (ragged, odd count)
        dict(name="linear features", op="linear", way="fwd", dtype="bf16", n=1970003, groups=4, k=64, m=256, skew=0.1),
        # experts' tokens, unevenly spread, as a mixture layer's router leaves them
        dict(name="linear experts", op="linear", way="fwd", dtype="bf16", n=40009, groups=32, k=1024, m=2048, skew=1.0),
        # fp32 rows of eight merged tables
        dict(name="linear fp32 rows", op="linear", way="fwd", dtype="f32", n=65536, groups=8, k=32, m=128, skew=0.3),
        # the gradients of an expert layer: inputs kept as they were
        dict(name="linear gradients", op="linear", way="bwd", dtype="bf16", n=65537, groups=16, k=512, m=1024, skew=1.0),
        # the gradients of the token block of a whole jagged batch, inputs kept in 8 bits
        dict(name="linear gradients, 8 bits", op="linear", way="bwd8", dtype="bf16", n=490011, groups=4, k=256, m=512, skew=0.3),
        # a few tokens while serving
        dict(name="norm 16 tokens", op="norm", way="fwd", dtype="bf16", kind="rms", gate="silu", n=16, groups=1, d=512, skew=0.0),
        # every token of a jagged batch, the next product's input kept in 8 bits
        dict(name="norm forward", op="norm", way="fwd8", dtype="bf16", kind="rms", gate="silu", n=490011, groups=4, d=512, skew=0.3),
        # layer norm with one set of parameters per group of tokens
        dict(name="norm gradients", op="norm", way="bwd", dtype="bf16", kind="layer", gate="sigmoid", n=200003, groups=8, d=1024, skew=1.0),
        # the same block's backward from checkpoints in 8 bits
        dict(name="norm gradients, 8 bits", op="norm", way="bwd8", dtype="bf16", kind="rms", gate="silu", n=490011, groups=4, d=512, skew=0.3),
        # the looked-up rows of a jagged batch, kept in 8 bits and read back
        dict(name="pack rows", op="pack", way="round trip", dtype="bf16", n=1970003, d=64),
        # a small fp32 activation whose last block is not full
        dict(name="pack odd", op="pack", way="round trip", dtype="f32", n=97, d=200),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["linear", "linear", "norm", "norm", "pack"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    groups = rng.choice([1, 2, 4, 5, 8, 13, 16, 32, 61])
    skew = round(rng.uniform(0.0, 1.0), 3)
    if op == "linear":
        way = rng.choice(["fwd", "bwd", "bwd8"])
        if dtype == "f32":
            k, m = rng.choice([16, 20, 32, 64, 128]), log(16, 256)
        else:
            k, m = (log(16, 1024), log(16, 2048)) if rng.random() < 0.3 else (8 * log(2, 128), 8 * log(2, 256))
        # at most about the gradients of the largest listed case, and odd widths at most a tenth of it
        most = 1.6e11 if way == "fwd" else 2.4e11
        if dtype == "f32" or k % 8 or m % 8:
            most /= 10
        top = most / ((2 if way == "fwd" else 4) * k * m)
        return dict(op=op, way=way, dtype=dtype, n=max(1, min(log(1, 1970003), int(top))), groups=groups, k=k, m=m, skew=skew)
    if op == "norm":
        d = rng.choice([16, 50, 64, 128, 200, 256, 512, 777, 1024, 2048])
        n = max(1, min(log(1, 1970003), int(2.0e8 / d)))
        way = rng.choice(["fwd", "fwd8", "bwd", "bwd8"])
        return dict(op=op, way=way, dtype=dtype, kind=rng.choice(["rms", "layer"]), gate=rng.choice(["none", "linear", "sigmoid", "silu"]),
                    n=n, groups=groups, d=d, skew=skew)
    d = rng.choice([16, 31, 32, 64, 100, 128, 512, 1024, 2047])
    return dict(op=op, way="round trip", dtype=dtype, n=max(1, min(log(1, 1970003), int(1.2e8 / d))), d=d)


def work(case):
    c, n = case, case["n"]
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "linear":
        k, m, g = c["k"], c["m"], min(c["groups"], n)
        if c["way"] == "fwd":
            return {"bytes": e * (n * k + n * m + g * k * m), "flops": 2 * n * k * m}
        x = n * (k + -(-k // BLOCK)) if c["way"] == "bwd8" else e * n * k
        return {"bytes": x + e * (n * m + g * k * m + n * k) + 4 * c["groups"] * k * m, "flops": 4 * n * k * m}
    d = c["d"]
    packed = n * (d + -(-d // BLOCK))
    if c["op"] == "pack":
        return {"bytes": 2 * e * n * d + 2 * packed, "flops": 4 * n * d}
    rows = 4 if c["gate"] == "none" else 5  # x, y, gate in; z, h out
    if c["way"] in ("fwd", "fwd8"):
        more = packed + packed + 2 * n * d if c["way"] == "fwd8" else 0  # the checkpoint written, read and spread again
        return {"bytes": rows * e * n * d + more, "flops": 20 * n * d}
    saved = rows - 2  # y, gate, z
    kept = saved * packed if c["way"] == "bwd8" else saved * e * n * d
    return {"bytes": kept + (2 + saved) * e * n * d, "flops": 40 * n * d}  # dz, dh in; dx, dy, dgate out


# ---- inputs -----------------------------------------------------------------------------------------------------------

def _sizes(case, seed):
    """Rows per group: about even for skew 0, some groups empty and a few long for skew 1."""
    n, groups = case["n"], case["groups"]
    rng = random.Random(1000003 * seed + n)
    if n < 4 * groups:
        sizes = [0] * groups
        for _ in range(n):
            sizes[rng.randrange(groups)] += 1
        return sizes
    share = [math.exp(1.2 * case["skew"] * rng.gauss(0.0, 1.0)) for _ in range(groups)]
    if case["skew"] >= 0.9 and groups > 8:
        share[rng.randrange(1, groups)] = 0.0
    cuts, run, total = [0], 0.0, sum(share)
    for s in share:
        run += s
        cuts.append(min(n, int(round(n * run / total))))
    cuts[-1] = n
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _pack(x):
    """Codes int8 [n, d] and exponent bytes [n, ceil(d / 32)] of the 8-bit form of x."""
    n, d = x.shape
    nb = -(-d // BLOCK)
    v = torch.zeros(n, nb * BLOCK, device=x.device, dtype=torch.float32)
    v[:, :d] = x
    v = v.view(n, nb, BLOCK)
    top = v.abs().amax(2)
    f, p = torch.frexp(top)
    e = torch.where(f <= 127 / 128, p - 7, p - 6).to(torch.int32)
    e = torch.where(top == 0, E_MIN, e).clamp(E_MIN, E_MAX)
    inv = ((127 - e) << 23).view(torch.float32)
    q = torch.round(v * inv[:, :, None]).clamp(-127, 127)
    bad = ~torch.isfinite(top)
    q = torch.where(bad[:, :, None], 0.0, q)
    byte = torch.where(bad, 255, e + 127)
    return q.view(n, nb * BLOCK)[:, :d].to(torch.int8).contiguous(), byte.to(torch.uint8)


def _unpack(codes, exps, dtype):
    e = exps.to(torch.int32)
    s = torch.where(e == 255, float("nan"), (e << 23).view(torch.float32))
    return (codes.to(torch.float32) * s.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]).to(dtype)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = TORCH[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)

    s = {"case": c}
    n = c["n"]
    if c["op"] == "pack":
        # activations: most values of order one, a few columns much larger
        s["x"] = (torch.randn(n, c["d"], generator=gen, device=DEV)
                  * torch.exp(0.7 * torch.randn(1, c["d"], generator=gen, device=DEV))).to(dt)
        return s
    sizes = _sizes(c, seed)
    off = [0]
    for z in sizes:
        off.append(off[-1] + z)
    s["offsets"] = torch.tensor(off, dtype=torch.int64, device=DEV)
    s["longest"] = max(sizes)
    if c["op"] == "linear":
        s["w"] = normal(c["groups"], c["m"], c["k"], scale=c["k"] ** -0.5)
        x = normal(n, c["k"])
        if c["way"] == "bwd8":
            s["x8"] = _pack(x)
        else:
            s["x"] = x
        if c["way"] != "fwd":
            s["dy"] = normal(n, c["m"])
        if own:
            import update_merged_table_gb300 as mt
            s["handle"] = mt.GroupedLinear(c["groups"], c["k"], c["m"], dtype=c["dtype"])
        return s
    d, g = c["d"], c["groups"]
    gated = c["gate"] != "none"
    biased = c["kind"] == "layer"

    def param(mean, spread):
        return mean + spread * torch.randn(g, d, generator=gen, device=DEV)

    s["post_weight"], s["pre_weight"] = param(1.0, 0.2), param(1.0, 0.2)
    s["post_bias"] = param(0.0, 0.1) if biased else None
    s["pre_bias"] = param(0.0, 0.1) if biased else None
    s["scale"] = param(0.5, 0.1)
    y, u, z = normal(n, d, scale=2.0), normal(n, d) if gated else None, normal(n, d, scale=1.5)
    if c["way"] in ("fwd", "fwd8"):
        s["x"], s["y"], s["u"] = z, y, u
    else:
        s["dz"], s["dh"] = normal(n, d), normal(n, d)
        if c["way"] == "bwd8":
            s["y8"], s["z8"], s["u8"] = _pack(y), _pack(z), _pack(u) if gated else None
        else:
            s["y"], s["u"], s["z"] = y, u, z
    if own:
        import update_merged_table_gb300 as mt
        s["handle"] = mt.GatedNorm(d, num_groups=g, kind=c["kind"], gate=c["gate"], eps=EPS, dtype=c["dtype"])
    return s


EPS = 1e-6


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "linear":
        return _plain_linear(state)
    if op == "norm":
        return _plain_norm(state)
    x = state["x"]
    return _unpack(*_pack(x), x.dtype)


def _run_own(s):
    import update_merged_table_gb300 as mt
    c = s["case"]
    if c["op"] == "pack":
        return mt.unpack8(mt.pack8(s["x"]), s["x"].dtype)
    if c["op"] == "linear":
        if c["way"] == "fwd":
            return s["handle"].forward(s["x"], s["w"], s["offsets"])
        x = mt.Packed8(*s["x8"]) if c["way"] == "bwd8" else s["x"]
        dx, dw = s["handle"].backward(s["dy"], x, s["w"], s["offsets"])
        return {"dx": dx, "dw": dw}
    p = mt.NormParams(s["post_weight"], s["post_bias"], s["scale"], s["pre_weight"], s["pre_bias"])
    if c["way"] == "fwd":
        r = s["handle"].forward(s["x"], s["y"], s["u"], p, s["offsets"])
        return {"z": r.z, "h": r.h}
    if c["way"] == "fwd8":
        r = s["handle"].forward(s["x"], s["y"], s["u"], p, s["offsets"], pack="h")
        return {"z": r.z, "h": r.h, "h8": mt.unpack8(r.packed["h"], torch.bfloat16)}
    if c["way"] == "bwd8":
        y, z = mt.Packed8(*s["y8"]), mt.Packed8(*s["z8"])
        u = mt.Packed8(*s["u8"]) if s["u8"] is not None else None
    else:
        y, u, z = s["y"], s["u"], s["z"]
    r = s["handle"].backward(s["dz"], s["dh"], y, u, z, p, s["offsets"])
    return _named(r.dx, r.dy, r.du, r.params.post_weight, r.params.post_bias, r.params.scale, r.params.pre_weight, r.params.pre_bias)


def _named(*v):
    names = ("dx", "dy", "du", "dpost_weight", "dpost_bias", "dscale", "dpre_weight", "dpre_bias")
    return {k: x for k, x in zip(names, v) if x is not None}


def _groups(s, n):
    """The group of each row and its place in it."""
    rows = torch.arange(n, device=DEV)
    g = torch.searchsorted(s["offsets"][1:], rows, right=True)
    return g, rows - s["offsets"][g]


def _plain_linear(s):
    c, n, off = s["case"], s["case"]["n"], s["offsets"]
    dt = TORCH[c["dtype"]]
    at = off[:-1, None] + torch.arange(s["longest"], device=DEV)
    live = (at < off[1:, None])[:, :, None]
    at = at.clamp(max=n - 1)
    g, place = _groups(s, n)
    w = s["w"].float()
    x = (_unpack(*s["x8"], torch.float32) if c["way"] == "bwd8" else s["x"].float())[at] * live
    if c["way"] == "fwd":
        return torch.matmul(x, w.transpose(1, 2))[g, place].to(dt)
    dy = s["dy"].float()[at] * live
    return {"dx": torch.matmul(dy, w)[g, place].to(dt), "dw": torch.matmul(dy.transpose(1, 2), x)}


def _norm(v, kind):
    """The normalised row and the inverse of its deviation."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    return v * r, r


def _norm_grad(dvh, vh, r, kind):
    d = dvh - vh * (dvh * vh).mean(1, keepdim=True)
    if kind == "layer":
        d = d - dvh.mean(1, keepdim=True)
    return d * r


def _gate(u, gate):
    """The gate's factor and its derivative."""
    if gate == "none":
        return 1.0, None
    if gate == "linear":
        return u, torch.ones_like(u)
    p = torch.sigmoid(u)
    if gate == "sigmoid":
        return p, p * (1 - p)
    return u * p, p * (1 + u * (1 - p))


def _plain_norm(s):
    c, n, dt = s["case"], s["case"]["n"], TORCH[s["case"]["dtype"]]
    kind, gate = c["kind"], c["gate"]
    g, _ = _groups(s, n)
    scale, pw, qw = s["scale"][g], s["post_weight"][g], s["pre_weight"][g]
    pb = s["post_bias"][g] if s["post_bias"] is not None else 0.0
    qb = s["pre_bias"][g] if s["pre_bias"] is not None else 0.0
    if c["way"] in ("fwd", "fwd8"):
        yh, _ = _norm(s["y"].float(), kind)
        a, _ = _gate(s["u"].float() if s["u"] is not None else None, gate)
        z = s["x"].float() + scale * (pw * yh + pb) * a
        h = qw * _norm(z, kind)[0] + qb
        out = {"z": z.to(dt), "h": h.to(dt)}
        if c["way"] == "fwd8":
            out["h8"] = _unpack(*_pack(out["h"]), torch.bfloat16)
        return out
    if c["way"] == "bwd8":
        y, z = _unpack(*s["y8"], torch.float32), _unpack(*s["z8"], torch.float32)
        u = _unpack(*s["u8"], torch.float32) if s["u8"] is not None else None
    else:
        y, z, u = s["y"].float(), s["z"].float(), s["u"].float() if s["u"] is not None else None
    dz, dh = s["dz"].float(), s["dh"].float()
    zh, rz = _norm(z, kind)
    d = dz + _norm_grad(dh * qw, zh, rz, kind)
    yh, ry = _norm(y, kind)
    t = pw * yh + pb
    a, da = _gate(u, gate)
    dt_ = d * scale * a
    dy = _norm_grad(dt_ * pw, yh, ry, kind)
    du = (d * scale * t * da).to(dt) if u is not None else None
    hot = (g[None, :] == torch.arange(c["groups"], device=DEV)[:, None]).float()  # sums over each group's rows

    def total(v):
        return torch.matmul(hot, v)

    biased = s["post_bias"] is not None
    return _named(d.to(dt), dy.to(dt), du, total(dt_ * yh), total(dt_) if biased else None, total(d * t * a), total(dh * zh),
                  total(dh) if biased else None)


# ---- the definition in 64 bits ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]

    def wide(name):
        if s.get(name) is not None:
            return s[name].double()
        if s.get(name + "8") is not None:
            codes, exps = s[name + "8"]
            power = torch.pow(2.0, exps.double() - 127.0)
            columns = torch.arange(codes.shape[1], device=DEV) // BLOCK
            return codes.double() * power[:, columns]
        return None

    if c["op"] == "pack":
        return wide("x")  # the values that the checkpoint stands in for
    bounds = s["offsets"].tolist()
    spans = list(zip(bounds, bounds[1:]))
    if c["op"] == "linear":
        x, w = wide("x"), s["w"].double()
        if c["way"] == "fwd":
            return torch.cat([x[a:b] @ w[g].T for g, (a, b) in enumerate(spans)])
        dy = wide("dy")
        return {"dx": torch.cat([dy[a:b] @ w[g] for g, (a, b) in enumerate(spans)]),
                "dw": torch.stack([dy[a:b].T @ x[a:b] for a, b in spans])}
    gates = {"linear": lambda v: v, "sigmoid": torch.sigmoid, "silu": lambda v: v / (1 + torch.exp(-v))}

    def normed(v):
        if c["kind"] == "layer":
            return (v - v.mean(1, keepdim=True)) / torch.sqrt(v.var(1, unbiased=False, keepdim=True) + EPS)
        return v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)

    def after(y, u, g, p):
        t = p["post_weight"][g] * normed(y)
        if p["post_bias"] is not None:
            t = t + p["post_bias"][g]
        t = p["scale"][g] * t
        return t if u is None else t * gates[c["gate"]](u)

    def before(z, g, p):
        h = p["pre_weight"][g] * normed(z)
        return h if p["pre_bias"] is None else h + p["pre_bias"][g]

    keys = ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")
    p = {k: wide(k) for k in keys}
    y, u = wide("y"), wide("u")
    if c["way"] in ("fwd", "fwd8"):
        x = wide("x")
        z = torch.cat([x[a:b] + after(y[a:b], None if u is None else u[a:b], g, p) for g, (a, b) in enumerate(spans)])
        h = torch.cat([before(z[a:b], g, p) for g, (a, b) in enumerate(spans)])
        return {"z": z, "h": h, "h8": h} if c["way"] == "fwd8" else {"z": z, "h": h}
    z, dz, dh = wide("z"), wide("dz"), wide("dh")
    rows = {"dx": [], "dy": [], "du": []}
    for k in keys:
        if p[k] is not None:
            p[k].requires_grad_(True)
    sums = {k: torch.zeros_like(p[k]) for k in keys if p[k] is not None}
    for g, (a0, b0) in enumerate(spans):
        for a in range(a0, b0, 65536):
            b = min(b0, a + 65536)
            zz = z[a:b].detach().requires_grad_(True)
            yy = y[a:b].detach().requires_grad_(True)
            uu = None if u is None else u[a:b].detach().requires_grad_(True)
            pre = [k for k in ("pre_weight", "pre_bias") if p[k] is not None]
            got = torch.autograd.grad(before(zz, g, p), [zz] + [p[k] for k in pre], dh[a:b])
            d = dz[a:b] + got[0]
            post = [k for k in ("post_weight", "post_bias", "scale") if p[k] is not None]
            leaves = [yy] + ([uu] if uu is not None else [])
            more = torch.autograd.grad(after(yy, uu, g, p), leaves + [p[k] for k in post], d)
            rows["dx"].append(d)
            rows["dy"].append(more[0])
            if uu is not None:
                rows["du"].append(more[1])
            for k, v in zip(pre + post, got[1:] + more[len(leaves):]):
                sums[k] += v
    whole = [torch.cat(v) if v else None for v in rows.values()]
    return _named(*whole, *(sums.get(k) for k in ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")))

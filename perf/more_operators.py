"""What follows the dense block's products: the cases that its feed-forward part and the losses over a vocabulary are measured on.

Three operators:

* ``gated``: the gated feed-forward part of a block, both projections, the activation and the product in one pass over ragged
  groups of rows (h = (Wy x) * act(Wu x)), and its gradients, with nothing kept from the forward but x.
* ``cross``: softmax cross entropy of rows against a large vocabulary (items, or the rows of a batch's keys), logits never
  kept, with the gradients of the rows and of the vocabulary.  Rows with a negative target are left out.
* ``distill``: the divergence from a teacher that is known by its top logits, over the same vocabulary, with its gradients.

Widths and counts follow the repository's workloads: 16 to 128 columns per table row, vocabularies of 10^4 to 3 * 10^5 keys,
thousands of users and tens of thousands of tokens; block widths of 256 to 2048 are generic.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token per request, each with its own expert: latency and the experts' weights
        dict(name="gated 8 tokens", op="gated", way="fwd", dtype="bf16", gate="silu", n=8, groups=8, k=512, m=1024, skew=0.0),
        # every token of a quarter of a jagged batch, four features with their own weights
        dict(name="gated features", op="gated", way="fwd", dtype="bf16", gate="silu", n=122503, groups=4, k=256, m=512, skew=0.3),
        # the gradients of a layer of uneven experts, products computed again
        dict(name="gated experts, gradients", op="gated", way="bwd", dtype="bf16", gate="silu", n=40009, groups=32, k=1024, m=2048, skew=1.0),
        # a small fp32 tower with widths that no vector divides
        dict(name="gated fp32 odd, gradients", op="gated", way="bwd", dtype="f32", gate="gelu", n=5003, groups=5, k=100, m=333, skew=0.5),
        # a few requests scored against every item of a table
        dict(name="cross 16 rows", op="cross", way="fwd", dtype="bf16", n=16, v=100003, d=256, masked=0.0, smoothing=0.0, z_loss=0.0),
        # a training step over an item vocabulary
        dict(name="cross step", op="cross", way="both", dtype="bf16", n=8192, v=100003, d=512, masked=0.1, smoothing=0.0, z_loss=1e-4),
        # the vocabulary is the table's rows of a jagged batch's keys
        dict(name="cross table rows", op="cross", way="both", dtype="bf16", n=16384, v=98001, d=64, masked=0.0, smoothing=0.0, z_loss=0.0),
        # long sequences of which half of the tokens carry no target
        dict(name="cross half masked", op="cross", way="both", dtype="bf16", n=65537, v=16384, d=256, masked=0.5, smoothing=0.1, z_loss=0.0),
        # fp32 rows
        dict(name="cross fp32", op="cross", way="both", dtype="f32", n=2048, v=10007, d=128, masked=0.2, smoothing=0.1, z_loss=1e-4),
        # a few rows' divergence while a student is watched, odd sizes
        dict(name="distill 37 rows", op="distill", way="fwd", dtype="bf16", n=37, v=32771, d=320, top=8, scale=1.0),
        # a distillation step
        dict(name="distill step", op="distill", way="both", dtype="bf16", n=4096, v=131072, d=1024, top=64, scale=0.5),
        # fp32 rows of a small table
        dict(name="distill fp32", op="distill", way="both", dtype="f32", n=1501, v=10007, d=64, top=33, scale=1.0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["gated", "cross", "cross", "distill"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "gated":
        way = rng.choice(["fwd", "bwd"])
        groups = rng.choice([1, 2, 4, 5, 8, 13, 16, 32, 61])
        k, m = (log(16, 1024), log(16, 2048)) if rng.random() < 0.3 else (8 * log(2, 128), 8 * log(2, 256))
        most = (1e12 if dtype == "bf16" else 4e10) / ((4 if way == "fwd" else 12) * k * m)
        return dict(op=op, way=way, dtype=dtype, gate=rng.choice(["linear", "sigmoid", "silu", "gelu"]), n=max(1, min(log(1, 490011), int(most))),
                    groups=groups, k=k, m=m, skew=round(rng.uniform(0.0, 1.0), 3))
    d = log(16, 1024) if rng.random() < 0.3 else 8 * log(2, 128)
    v = log(2, 300000)
    way = rng.choice(["fwd", "both", "both"])
    flops = 2 if way == "fwd" else 6
    most = min((3e12 if dtype == "bf16" else 6e10) / (flops * d * v), 2e9 / v)  # 2e9: the plain form's logits
    n = max(1, min(log(1, 65537), int(most)))
    if op == "cross":
        return dict(op=op, way=way, dtype=dtype, n=n, v=v, d=d, masked=rng.choice([0.0, 0.1, 0.5, 0.9]), smoothing=rng.choice([0.0, 0.0, 0.1]),
                    z_loss=rng.choice([0.0, 1e-4]))
    return dict(op=op, way=way, dtype=dtype, n=n, v=v, d=d, top=min(log(1, 128), v), scale=rng.choice([1.0, 0.5, 0.25]))


def work(case):
    c, n = case, case["n"]
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "gated":
        k, m, g = c["k"], c["m"], min(c["groups"], n)
        if c["way"] == "fwd":
            return {"bytes": e * (n * k + n * m + 2 * g * k * m), "flops": 4 * n * k * m}
        return {"bytes": e * (2 * n * k + n * m + 2 * g * k * m + 2 * c["groups"] * k * m), "flops": 12 * n * k * m}
    v, d = c["v"], c["d"]
    live = n - _masked_rows(c) if c["op"] == "cross" else n
    side = 4 if c["op"] == "cross" else 8 * c["top"]
    if c["way"] == "fwd":
        return {"bytes": e * (live * d + v * d) + n * (side + 8), "flops": 2 * live * v * d}
    return {"bytes": e * (live * d + n * d + 2 * v * d) + n * (side + 12), "flops": 6 * live * v * d}


def _masked_rows(c):
    return int(c["masked"] * c["n"])


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


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = TORCH[c["dtype"]]
    n = c["n"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=DEV) * scale

    s = {"case": c}
    if c["op"] == "gated":
        sizes = _sizes(c, seed)
        off = [0]
        for z in sizes:
            off.append(off[-1] + z)
        s["offsets"] = torch.tensor(off, dtype=torch.int64, device=DEV)
        s["longest"] = max(sizes)
        s["x"] = normal(n, c["k"]).to(dt)
        s["w"] = normal(c["groups"], 2 * c["m"], c["k"], scale=c["k"] ** -0.5).to(dt)
        if c["way"] == "bwd":
            s["dh"] = normal(n, c["m"]).to(dt)
        if own:
            import update_merged_table_gb300 as mt
            s["handle"] = mt.GatedLinear(c["groups"], c["k"], c["m"], gate=c["gate"], dtype=c["dtype"])
        return s
    v, d = c["v"], c["d"]
    w = normal(v, d, scale=1.5 * d ** -0.5)
    # popular items are targets more often than others
    hit = (v * torch.rand(n, generator=gen, device=DEV).square()).long().clamp_(max=v - 1)
    # a student that has learnt something: the rows lean towards their targets
    s["x"] = (normal(n, d) + 1.2 * w[hit]).to(dt)
    s["w"] = w.to(dt)
    s["dloss"] = (0.5 + torch.rand(n, generator=gen, device=DEV)) / n
    if c["op"] == "cross":
        out = torch.randperm(n, generator=gen, device=DEV)[:_masked_rows(c)]
        s["targets"] = hit.to(torch.int32)
        s["targets"][out] = -1
        if own:
            import update_merged_table_gb300 as mt
            s["handle"] = mt.CrossEntropy(v, d, smoothing=c["smoothing"], z_loss=c["z_loss"], dtype=c["dtype"])
        return s
    top = c["top"]
    ids = torch.randint(0, v, (n, top), generator=gen, device=DEV, dtype=torch.int64)
    ids[:, 0] = hit
    # some teachers kept fewer than `top`: the rest of the row is -1
    kept = torch.randint(1, 4 * top + 1, (n, 1), generator=gen, device=DEV)
    s["ids"] = torch.where(torch.arange(top, device=DEV)[None, :] < kept, ids, -1).to(torch.int32)
    s["teacher"] = (2.0 * torch.randn(n, top, generator=gen, device=DEV) + 3.0).sort(dim=1, descending=True).values
    if own:
        import update_merged_table_gb300 as mt
        s["handle"] = mt.Distillation(v, d, top, scale=c["scale"], dtype=c["dtype"])
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own_gated(state) if op == "gated" else _own_loss(state)
    return _plain_gated(state) if op == "gated" else _plain_loss(state)


def _own_gated(s):
    if s["case"]["way"] == "fwd":
        return s["handle"].forward(s["x"], s["w"], s["offsets"])
    dx, dw = s["handle"].backward(s["dh"], s["x"], s["w"], s["offsets"])
    return {"dx": dx, "dw": dw}


def _own_loss(s):
    of = (s["targets"],) if s["case"]["op"] == "cross" else (s["ids"], s["teacher"])
    r = s["handle"].forward(s["x"], s["w"], *of)
    if s["case"]["way"] == "fwd":
        return {"loss": r.loss, "lse": r.lse}
    dx, dw = s["handle"].backward(s["dloss"], s["x"], s["w"], *of, r.lse)
    return {"loss": r.loss, "lse": r.lse, "dx": dx, "dw": dw}


def _gate(u, gate):
    """The gate's factor and its derivative."""
    if gate == "linear":
        return u, torch.ones_like(u)
    if gate == "gelu":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        p = 1.0 / (1.0 + torch.exp(-c * (u + 0.044715 * u * u * u)))
        return u * p, p + u * p * (1.0 - p) * c * (1.0 + 3.0 * 0.044715 * u * u)
    p = 1.0 / (1.0 + torch.exp(-u))
    return (p, p * (1.0 - p)) if gate == "sigmoid" else (u * p, p * (1.0 + u * (1.0 - p)))


def _plain_gated(s):
    c, n, m, dt, off = s["case"], s["case"]["n"], s["case"]["m"], TORCH[s["case"]["dtype"]], s["offsets"]
    at = off[:-1, None] + torch.arange(s["longest"], device=DEV)  # every group padded to the longest
    live = (at < off[1:, None])[:, :, None]
    at = at.clamp(max=n - 1)
    rows = torch.arange(n, device=DEV)
    g = torch.searchsorted(off[1:], rows, right=True)
    place = rows - off[g]
    x, w = s["x"].float()[at] * live, s["w"].float()
    t = torch.matmul(x, w.transpose(1, 2))
    y, u = t[:, :, :m], t[:, :, m:]
    a, da = _gate(u, c["gate"])
    if c["way"] == "fwd":
        return (y * a)[g, place].to(dt)
    dh = s["dh"].float()[at] * live
    d = torch.cat([dh * a, dh * y * da], 2)
    return {"dx": torch.matmul(d, w)[g, place].to(dt), "dw": torch.matmul(d.transpose(1, 2), x).to(dt)}


def _teacher(s, wide):
    """Where the rows' kept entries are, and the teacher's distribution over them (zero elsewhere)."""
    there = s["ids"] >= 0
    logits = torch.where(there, s["teacher"].to(wide) * s["case"]["scale"], -math.inf)
    e = torch.where(there, torch.exp(logits - logits.amax(1, keepdim=True)), 0.0)
    return there, s["ids"].long().clamp(min=0), e / e.sum(1, keepdim=True)


def _plain_loss(s):
    c, dt = s["case"], TORCH[s["case"]["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    v, scale, z_loss, smoothing = c["v"], c.get("scale", 1.0), c.get("z_loss", 0.0), c.get("smoothing", 0.0)
    z = torch.matmul(x, w.T)
    if scale != 1.0:
        z *= scale
    top = z.amax(1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    if c["op"] == "cross":
        live = s["targets"] >= 0
        at = s["targets"].long().clamp(min=0)[:, None]
        share = (1.0 - smoothing) * live[:, None].float()
        loss = lse - (1.0 - smoothing) * z.gather(1, at)[:, 0]
        if smoothing:
            loss = loss - smoothing / v * z.sum(1)
        loss = torch.where(live, loss + z_loss * lse * lse, 0.0)
    else:
        there, at, share = _teacher(s, torch.float32)
        live = there.any(1)
        loss = lse + torch.where(share > 0, share * (torch.log(share) - z.gather(1, at)), 0.0).sum(1)
        loss = torch.where(live, loss, 0.0)
    out = {"loss": loss, "lse": torch.where(live, lse, 0.0)}
    if c["way"] == "fwd":
        return out
    del z
    p *= (1.0 + 2.0 * z_loss * lse)[:, None] / total
    if smoothing:
        p -= smoothing / v
    p.scatter_add_(1, at, -share)
    p *= torch.where(live, s["dloss"] * scale, 0.0)[:, None]
    out["dx"], out["dw"] = torch.matmul(p, w).to(dt), torch.matmul(p.T, x * live[:, None]).to(dt)
    return out


# ---- the definition in 64 bits ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_gated(s) if case["op"] == "gated" else _exact_loss(s)


def _exact_gated(s):
    c, m = s["case"], s["case"]["m"]
    gates = {"linear": lambda v: v, "sigmoid": torch.sigmoid, "silu": lambda v: v * torch.sigmoid(v),
             "gelu": lambda v: 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))}
    bounds = s["offsets"].tolist()
    h, dx, dw = [], [], []
    for g, (a, b) in enumerate(zip(bounds, bounds[1:])):
        x = s["x"][a:b].double().requires_grad_(True)
        w = s["w"][g].double().requires_grad_(True)
        out = (x @ w[:m].T) * gates[c["gate"]](x @ w[m:].T)
        if c["way"] == "fwd":
            h.append(out.detach())
            continue
        got = torch.autograd.grad(out, (x, w), s["dh"][a:b].double())
        dx.append(got[0])
        dw.append(got[1])
    return torch.cat(h) if c["way"] == "fwd" else {"dx": torch.cat(dx), "dw": torch.stack(dw)}


def _exact_loss(s):
    c, n, v = s["case"], s["case"]["n"], s["case"]["v"]
    w = s["w"].double()
    scale = c.get("scale", 1.0)
    loss, lse = torch.zeros(n, device=DEV, dtype=torch.float64), torch.zeros(n, device=DEV, dtype=torch.float64)
    dx, dw = torch.zeros(n, c["d"], device=DEV, dtype=torch.float64), torch.zeros_like(w)
    if c["op"] == "cross":
        rows = torch.nonzero(s["targets"] >= 0)[:, 0]
    else:
        rows = torch.nonzero((s["ids"] >= 0).any(1))[:, 0]
    step = max(1, 2 ** 28 // v)
    for a in range(0, rows.numel(), step):
        at = rows[a:a + step]
        x = s["x"][at].double()
        z = scale * (x @ w.T)
        log_sum = torch.logsumexp(z, 1)
        if c["op"] == "cross":
            q = torch.full_like(z, c["smoothing"] / v)
            q.scatter_add_(1, s["targets"][at].long()[:, None], torch.full((at.numel(), 1), 1.0 - c["smoothing"], device=DEV, dtype=torch.float64))
            loss[at] = -(q * (z - log_sum[:, None])).sum(1) + c["z_loss"] * log_sum ** 2
            more = 2.0 * c["z_loss"] * log_sum
        else:
            ids, logits = s["ids"][at].long(), scale * s["teacher"][at].double()
            t = torch.softmax(logits.masked_fill(ids < 0, -math.inf), 1)
            ids = torch.where(ids < 0, 0, ids)
            loss[at] = torch.special.xlogy(t, t).sum(1) - (t * (z.gather(1, ids) - log_sum[:, None])).sum(1)
            q = torch.zeros_like(z).scatter_add_(1, ids, t)
            more = 0.0 * log_sum
        lse[at] = log_sum
        if c["way"] == "fwd":
            continue
        dz = torch.softmax(z, 1) * (1.0 + more)[:, None] - q
        dz *= (scale * s["dloss"][at].double())[:, None]
        dx[at] = dz @ w
        dw += dz.T @ x
    return {"loss": loss, "lse": lse} if c["way"] == "fwd" else {"loss": loss, "lse": lse, "dx": dx, "dw": dw}

"""What is measured of the mixture-of-experts operators: the router with its
balance loss, counts and gradients; the dispatch of token rows into expert
groups and the weighted combine back, with their gradients; the Newton-Schulz
orthogonalisation of expert-weight updates.

Every pass is computed in plain torch operations in 32 bits, or with ``own``
set by the package's operators.  Shapes follow the package's benchmark
operands: 16384 tokens of 4096 features over 8 or 256 experts, expert weights
of 8192 x 5120.
"""
import math

import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token of one request passes the router while serving: latency
        dict(name="route_serve", op="route", tokens=1, experts=256, top_k=8, dtype="bf16", renorm=True, align=1,
             masked=False, limited=False, grad=False),
        # training batch, 8 experts, two per token: forward, losses and the logits' gradient
        dict(name="route_train_8", op="route", tokens=16384, experts=8, top_k=2, dtype="bf16", renorm=True, align=1,
             masked=False, limited=False, grad=True),
        # training batch over 256 fine-grained experts, padded sequences, fp32 logits, groups on multiples of 16
        dict(name="route_train_256", op="route", tokens=16384, experts=256, top_k=8, dtype="fp32", renorm=True, align=16,
             masked=True, limited=False, grad=True),
        # odd sizes; some experts unavailable to a token, some tokens with no expert left; weights not renormalised
        dict(name="route_odd", op="route", tokens=4099, experts=61, top_k=6, dtype="bf16", renorm=False, align=32,
             masked=True, limited=True, grad=True),
        # a decoding batch of 8 requests gets its experts' rows back, added to the residual stream
        dict(name="combine_serve", op="combine", tokens=8, width=5120, experts=256, top_k=8, dtype="bf16", align=1,
             masked=False, residual=True, grad=False),
        # training batch into the groups of 8 experts, and the gradient back to the tokens
        dict(name="dispatch_train", op="dispatch", tokens=16384, width=4096, experts=8, top_k=2, dtype="bf16", align=1,
             masked=False, residual=False, grad=True),
        # the same batch back from the experts, with the gradients of rows and weights
        dict(name="combine_train", op="combine", tokens=16384, width=4096, experts=8, top_k=2, dtype="bf16", align=16,
             masked=True, residual=False, grad=True),
        # odd width and token count in fp32, padded groups
        dict(name="dispatch_odd", op="dispatch", tokens=2049, width=1111, experts=13, top_k=3, dtype="fp32", align=16,
             masked=True, residual=False, grad=True),
        # one small square matrix (a shared projection): latency of the chain of products
        dict(name="muon_small", op="muon", count=1, rows=512, cols=512, dtype="fp32"),
        # odd matrices in fp32
        dict(name="muon_odd", op="muon", count=3, rows=1000, cols=777, dtype="fp32"),
        # the down projections of 32 fine-grained experts: tall matrices
        dict(name="muon_experts", op="muon", count=32, rows=2048, cols=768, dtype="bf16"),
        # one expert's weights at full size
        dict(name="muon_large", op="muon", count=1, rows=8192, cols=5120, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "muon"])
    if op == "muon":
        c = dict(op=op, count=_log(rng, 1, 32), rows=_log(rng, 64, 8192), cols=_log(rng, 64, 8192),
                 dtype=rng.choice(["bf16", "fp32"]))
        while _plain_flops(c) > 1.5e12:
            c["count"], c["rows"], c["cols"] = max(1, c["count"] // 2), c["rows"] * 3 // 4, c["cols"] * 3 // 4
        return c
    tokens, experts = _log(rng, 1, 16384), _log(rng, 4, 512)
    c = dict(op=op, tokens=tokens, experts=experts, top_k=rng.randint(1, min(8, experts)),
             dtype=rng.choice(["bf16", "fp32"]), align=rng.choice([1, 16, 32]), masked=rng.random() < 0.5,
             grad=rng.random() < 0.75)
    if op == "route":
        c.update(renorm=rng.random() < 0.5, limited=rng.random() < 0.25)
        return c
    c.update(width=_log(rng, 64, 8192), residual=op == "combine" and rng.random() < 0.5)
    if rng.random() < 0.5:  # model widths are mostly multiples of 64
        c["width"] = (c["width"] + 63) // 64 * 64
    while c["tokens"] * c["width"] * (1 + c["top_k"]) > 16384 * 4096 * 3:
        c["tokens"] = c["tokens"] // 2
    return c


def _plain_flops(case):
    m, n = sorted((case["rows"], case["cols"]))
    return case["count"] * STEPS * (4.0 * m * m * n + 2.0 * m ** 3)


def capacity(case):
    """Rows of the buffer that holds every group, whatever the router picks."""
    slots = case["tokens"] * case["top_k"]
    return slots + min(case["experts"], slots) * (case["align"] - 1)


# ---------------------------------------------------------------- inputs

def _token_mask(case, g):
    """Padded sequences: about a tenth of the tokens carry nothing."""
    if not case["masked"]:
        return None
    t, seq = case["tokens"], 512
    n = (t + seq - 1) // seq
    ends = torch.randint(seq * 4 // 5, seq + 1, (n, 1), generator=g, device="cuda")
    return (torch.arange(seq, device="cuda")[None, :] < ends).reshape(-1)[:t].contiguous()


def _logits(case, g):
    """Router logits: a common bias makes some experts more popular."""
    t, e = case["tokens"], case["experts"]
    x = 1.5 * torch.randn(t, e, generator=g, device="cuda")
    x = x + 0.5 * torch.randn(1, e, generator=g, device="cuda")
    if case.get("limited"):
        blocks = (e + 7) // 8
        off = torch.rand(t, blocks, generator=g, device="cuda") < 0.5
        off |= torch.rand(t, 1, generator=g, device="cuda") < 1 / 256
        x = x.masked_fill(off.repeat_interleave(8, 1)[:, :e], -math.inf)
    return x.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "muon":
        # a momentum buffer: gradients are products of per-token rows, whose
        # features have scales of their own; G = dY^T X over some tokens
        c, r, k = case["count"], case["rows"], case["cols"]
        t = min(2 * min(r, k), 4096)
        parts = []
        for _ in range(c):
            dy = torch.randn(t, r, generator=g, device="cuda") * torch.exp(torch.randn(t, 1, generator=g, device="cuda"))
            x = torch.randn(t, k, generator=g, device="cuda") * torch.exp(0.7 * torch.randn(1, k, generator=g, device="cuda"))
            parts.append((dy.t().contiguous() @ x * (1e-3 / math.sqrt(t))).to(dt))
        s["g"] = torch.stack(parts)
        return s
    t, k = case["tokens"], case["top_k"]
    s["mask"] = _token_mask(case, g)
    s["logits"] = _logits(case, g)
    if case["op"] == "route":
        if case["grad"]:
            s["grad_weights"] = torch.randn(t, k, generator=g, device="cuda") * 1e-2
            s["grad_losses"] = torch.tensor([1e-2, 1e-3], device="cuda")
        return s
    r = _route(s["logits"].float(), s["mask"], k, True, case["align"])
    s["ids"], s["weights"], s["rows"], s["counts"], s["offs"] = (r[n] for n in ("ids", "weights", "rows", "counts", "offs"))
    w, cap = case["width"], capacity(case)
    if case["op"] == "dispatch":
        s["x"] = torch.randn(t, w, generator=g, device="cuda").to(dt)
        if case["grad"]:
            s["grad_xg"] = (torch.randn(cap, w, generator=g, device="cuda") * 1e-2).to(dt)
    else:
        s["yg"] = torch.randn(cap, w, generator=g, device="cuda").to(dt)
        if case["residual"]:
            s["residual"] = torch.randn(t, w, generator=g, device="cuda").to(dt)
        if case["grad"]:
            s["grad_y"] = (torch.randn(t, w, generator=g, device="cuda") * 1e-2).to(dt)
    return s


# ---------------------------------------------------------------- plain forms (32 bits)

def _route(x, mask, k, renorm, align):
    t, e = x.shape
    live = (x > -math.inf).any(1)
    if mask is not None:
        live = live & mask
    n = live.sum()
    top = x.amax(1, keepdim=True)
    lse = (x - top).exp().sum(1).log() + top[:, 0]
    lse = torch.where(live, lse, math.inf)
    p = (x - lse[:, None]).exp()
    best, ids = torch.sort(x, dim=1, descending=True, stable=True)
    taken = (best[:, :k] > -math.inf) & live[:, None]
    ids = ids[:, :k]
    w = torch.where(taken, p.gather(1, ids), 0.0)
    if renorm:
        w = torch.where(taken, w / w.sum(1, keepdim=True), 0.0)
    hit = torch.zeros(t, e, dtype=torch.int32, device=x.device)
    hit.scatter_(1, ids, taken.int())
    before = hit.t().contiguous().cumsum(1).t() - hit
    counts = hit.sum(0)
    offs = ((counts + align - 1) // align * align).cumsum(0)
    starts = offs - (counts + align - 1) // align * align
    rows = before.gather(1, ids) + starts[ids]
    nf = n.clamp(min=1).float()
    mean_prob = p.sum(0) / nf
    f = counts.float() / (nf * k)
    losses = torch.stack([e * (f * mean_prob).sum(), torch.where(live, lse, 0.0).square().sum() / nf])
    i32 = torch.int32
    return {"ids": torch.where(taken, ids, -1).to(i32), "weights": w, "rows": torch.where(taken, rows, -1).to(i32),
            "counts": counts.to(i32), "offs": offs.to(i32), "mean_prob": mean_prob, "losses": losses, "lse": lse,
            "live": n.reshape(1).to(i32), "p": p}


def _route_backward(r, renorm, grad_weights, grad_losses):
    p, e, k = r["p"], r["p"].shape[1], r["ids"].shape[1]
    n = r["live"].clamp(min=1).float()
    taken = r["ids"] >= 0
    at = r["ids"].clamp(min=0).long()
    q = torch.where(taken, grad_weights, 0.0)
    if renorm:
        total = torch.where(taken, p.gather(1, at), 0.0).sum(1, keepdim=True)
        q = torch.where(taken, (q - (q * r["weights"]).sum(1, keepdim=True)) / total, 0.0)
    dp = (grad_losses[0] * e / (n * n * k) * r["counts"].float())[None, :].expand(p.shape[0], e).clone()
    dp.scatter_add_(1, at, q)
    z = torch.where(r["lse"] < math.inf, r["lse"], 0.0) * (2.0 * grad_losses[1] / n)
    return p * (dp - (p * dp).sum(1, keepdim=True) + z[:, None])


def _gather_rows(xg, rows):
    return torch.where((rows >= 0)[:, :, None], xg[rows.clamp(min=0).long()].float(), 0.0)


def _scatter_rows(values, rows, cap):
    """values (T, k, W) to their rows of a (cap, W) buffer of zeros."""
    out = torch.zeros(cap + 1, values.shape[2], dtype=torch.float32, device=values.device)
    out[torch.where(rows >= 0, rows, cap).long().reshape(-1)] = values.reshape(-1, values.shape[2])
    return out[:cap]


def _newton_schulz(g):
    a, b, c = COEFFICIENTS
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        m = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * m + c * (m @ m)) @ x
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


def _run_plain(s):
    c = s["case"]
    if c["op"] == "muon":
        return {"update": _newton_schulz(s["g"])}
    if c["op"] == "route":
        r = _route(s["logits"].float(), s["mask"], c["top_k"], c["renorm"], c["align"])
        out = {n: r[n] for n in ("ids", "weights", "rows", "counts", "offs", "mean_prob", "losses", "lse", "live")}
        if c["grad"]:
            d = _route_backward(r, c["renorm"], s["grad_weights"], s["grad_losses"])
            out["grad_logits"] = d.to(s["logits"].dtype)
        return out
    rows, cap = s["rows"], capacity(c)
    if c["op"] == "dispatch":
        x = s["x"]
        out = {"xg": _scatter_rows(x.float()[:, None, :].expand(-1, c["top_k"], -1), rows, cap).to(x.dtype)}
        if c["grad"]:
            out["grad_x"] = _gather_rows(s["grad_xg"], rows).sum(1).to(x.dtype)
        return out
    w = s["weights"]
    back = _gather_rows(s["yg"], rows)
    y = (back * w[:, :, None]).sum(1)
    if c["residual"]:
        y = y + s["residual"].float()
    out = {"y": y.to(s["yg"].dtype)}
    if c["grad"]:
        dy = s["grad_y"].float()
        out["grad_yg"] = _scatter_rows(dy[:, None, :] * w[:, :, None], rows, cap).to(s["yg"].dtype)
        out["grad_weights"] = (back * dy[:, None, :]).sum(2)
    return out


# ---------------------------------------------------------------- the package's operators

def _run_own(s):
    import mxfp8_quantization_moe_amd as mxq

    c = s["case"]
    if c["op"] == "muon":
        return {"update": mxq.muon_orthogonalize(s["g"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)}
    if c["op"] == "route":
        r = mxq.moe_route(s["logits"], c["top_k"], token_mask=s["mask"], renormalize=c["renorm"], align=c["align"])
        out = {"ids": r.ids, "weights": r.weights, "rows": r.rows, "counts": r.counts, "offs": r.offs,
               "mean_prob": r.mean_prob, "losses": r.losses, "lse": r.lse, "live": r.live}
        if c["grad"]:
            out["grad_logits"] = mxq.moe_route_backward(s["logits"], r, s["grad_weights"], s["grad_losses"])
        return out
    r = mxq.MoeRoute(ids=s["ids"], weights=s["weights"], rows=s["rows"], counts=s["counts"], offs=s["offs"],
                     align=c["align"])
    if c["op"] == "dispatch":
        out = {"xg": mxq.moe_dispatch(s["x"], r)}
        if c["grad"]:
            out["grad_x"] = mxq.moe_dispatch_backward(s["grad_xg"], r)
        return out
    out = {"y": mxq.moe_combine(s["yg"], r, residual=s.get("residual"))}
    if c["grad"]:
        out["grad_yg"], out["grad_weights"] = mxq.moe_combine_backward(s["grad_y"], s["yg"], r)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- work

def work(case):
    size = {"bf16": 2, "fp32": 4}[case["dtype"]]
    if case["op"] == "muon":
        # A and A^2 are symmetric: half of each product
        m, n = sorted((case["rows"], case["cols"]))
        return {"bytes": case["count"] * m * n * (size + 2),
                "flops": case["count"] * STEPS * (3.0 * m * m * n + 1.0 * m ** 3)}
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    slots = t * k
    if case["op"] == "route":
        # logits; ids, weights, rows; lse; the per-expert arrays.  Backward:
        # logits and their gradient, the slots' ids, weights and gradients
        nbytes = t * e * size + slots * 12 + t * 4 + e * 12 + (t if case["masked"] else 0)
        flops = t * e * 6.0
        if case["grad"]:
            nbytes += 2 * t * e * size + slots * 12 + t * 4
            flops += t * e * 8.0
        return {"bytes": nbytes, "flops": flops}
    w, cap = case["width"], capacity(case)
    side, group, plan = t * w * size, cap * w * size, slots * 4
    if case["op"] == "dispatch":
        nbytes, flops = side + group + plan, 0.0
        if case["grad"]:
            nbytes, flops = nbytes + slots * w * size + side + plan, slots * w * 1.0
        return {"bytes": nbytes, "flops": flops}
    nbytes = slots * w * size + side * (2 if case["residual"] else 1) + 2 * plan
    flops = slots * w * 2.0
    if case["grad"]:
        nbytes += side + slots * w * size + group + 3 * plan
        flops += slots * w * 3.0
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_route(logits, mask, k, renorm, grad_weights, grad_losses):
    import numpy as np

    l = logits.double().cpu().numpy()
    t, e = l.shape
    ok = np.ones(t, bool) if mask is None else mask.cpu().numpy().astype(bool)
    alive = ok & (l.max(1) > -np.inf)
    n = max(int(alive.sum()), 1)
    la = l[alive]
    ex = np.exp(la - la.max(1, keepdims=True))
    z = np.log(ex.sum(1)) + la.max(1)
    pa = ex / ex.sum(1, keepdims=True)
    pick = np.argsort(-la, axis=1, kind="stable")[:, :k]
    there = np.take_along_axis(la, pick, 1) > -np.inf
    pp = np.take_along_axis(pa, pick, 1) * there
    s = pp.sum(1, keepdims=True) if renorm else np.ones((len(la), 1))
    wa = pp / s
    counts = np.bincount(pick[there], minlength=e)
    mean = pa.sum(0) / n
    out = {"ids": None, "rows": None, "counts": None, "offs": None, "live": None}
    w = np.zeros((t, k))
    w[alive] = wa
    lse = np.full(t, np.inf)
    lse[alive] = z
    out.update(weights=w, lse=lse, mean_prob=mean,
               losses=np.array([e * (counts / (n * k) * mean).sum(), (z * z).sum() / n]))
    if grad_weights is not None:
        gw = grad_weights.double().cpu().numpy()[alive] * there
        gl = grad_losses.double().cpu().numpy()
        # dw_j/dp_i = ([i = j] - w_j) / s with renormalisation, [i = j] without
        q = (gw - (gw * wa).sum(1, keepdims=True)) / s if renorm else gw
        dp = np.tile(gl[0] * e * counts / (n * k) / n, (len(la), 1))
        for j in range(k):
            dp[np.arange(len(la)), pick[:, j]] += q[:, j] * there[:, j]
        d = np.zeros((t, e))
        d[alive] = pa * (dp - (dp * pa).sum(1, keepdims=True)) + pa * (gl[1] * 2 * z / n)[:, None]
        out["grad_logits"] = d
    return out


def _exact_muon(g):
    a, b, c = COEFFICIENTS
    outs = []
    for i in range(g.shape[0]):
        x = g[i].double()
        x = x / (torch.linalg.vector_norm(x) + EPS)
        for _ in range(STEPS):
            if x.shape[0] <= x.shape[1]:
                m = x @ x.t().contiguous()
                x = a * x + b * (m @ x) + c * (m @ (m @ x))
            else:
                m = x.t().contiguous() @ x
                x = a * x + b * (x @ m) + c * ((x @ m) @ m)
        outs.append(x)
    return torch.stack(outs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "muon":
        return {"update": _exact_muon(s["g"])}
    if case["op"] == "route":
        return _exact_route(s["logits"], s["mask"], case["top_k"], case["renorm"], s.get("grad_weights"), s.get("grad_losses"))
    rows, k, cap = s["rows"].long(), case["top_k"], capacity(case)
    out = {}
    if case["op"] == "dispatch":
        x = s["x"].double()
        xg = torch.zeros(cap, x.shape[1], dtype=torch.float64, device="cuda")
        dx = torch.zeros_like(x)
        for j in range(k):
            on = rows[:, j] >= 0
            xg[rows[on, j]] = x[on]
            if case["grad"]:
                dx[on] += s["grad_xg"][rows[on, j]].double()
        out["xg"] = xg
        if case["grad"]:
            out["grad_x"] = dx
        return out
    w, yg = s["weights"].double(), s["yg"]
    y = s["residual"].double() if case["residual"] else torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
    dyg = torch.zeros(cap, case["width"], dtype=torch.float64, device="cuda") if case["grad"] else None
    dw = torch.zeros_like(w)
    for j in range(k):
        on = rows[:, j] >= 0
        back = yg[rows[on, j]].double()
        y[on] += w[on, j:j + 1] * back
        if case["grad"]:
            dy = s["grad_y"][on].double()
            dyg[rows[on, j]] = w[on, j:j + 1] * dy
            dw[on, j] = (back * dy).sum(1)
    out["y"] = y
    if case["grad"]:
        out.update(grad_yg=dyg, grad_weights=dw)
    return out

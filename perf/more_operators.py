"""What is measured of the experts' products: the matrix product of token
groups with their experts' weights with bias, activation, gate and residual in
its epilogue and its gradients, in bf16 and on MXFP8 operands, and a whole
mixture-of-experts layer for a few tokens.

Every pass is computed in plain torch operations in 32 bits, or with ``own``
set by the package's operators.  Shapes follow the package's benchmark
operands and examples: expert weights of 8192 x 5120 and 4096 x 4096, 16384
tokens over 8 experts, fine-grained experts of 2048 x 768.
"""
import math

import torch

own = False

BF16 = torch.bfloat16


def listed():
    return [
        # one token through a dense projection with everything in its epilogue: latency
        dict(name="linear_token", op="linear", rows=1, experts=1, width=4096, out=4096, act="gelu", gated=False,
             bias=True, residual=True, grad=False, skew=0.0),
        # a decoding batch already in its groups, two rows or so for each of 64 fine-grained experts
        dict(name="linear_decode", op="linear", rows=128, experts=64, width=2048, out=768, act="silu", gated=True,
             bias=False, residual=False, grad=False, skew=0.5),
        # a dense feed-forward's first product in training, forward and gradients
        dict(name="linear_dense", op="linear", rows=8192, experts=1, width=5120, out=8192, act="gelu", gated=False,
             bias=True, residual=False, grad=True, skew=0.0),
        # 16384 tokens in two slots each over 8 experts, gate and value projections in one product
        dict(name="linear_experts", op="linear", rows=32768, experts=8, width=4096, out=2048, act="silu", gated=True,
             bias=False, residual=False, grad=True, skew=0.3),
        # the down projections of 64 fine-grained experts: short sums, many groups
        dict(name="linear_fine", op="linear", rows=32768, experts=64, width=768, out=2048, act="none", gated=False,
             bias=True, residual=False, grad=True, skew=0.3),
        # odd sizes throughout, some experts without a row
        dict(name="linear_odd", op="linear", rows=6147, experts=13, width=1111, out=777, act="relu", gated=False,
             bias=True, residual=True, grad=True, skew=0.5),
        # expert weights at full size on MXFP8 operands, as the quantizers write them
        dict(name="mx_experts", op="linear_mx", rows=16384, experts=8, width=5120, out=8192, act="none", gated=False,
             bias=False, residual=False, skew=0.3),
        # gated fine-grained experts on MXFP8 operands, groups that end anywhere
        dict(name="mx_odd", op="linear_mx", rows=4099, experts=61, width=2080, out=744, act="silu", gated=True,
             bias=True, residual=False, skew=0.5),
        # one token of one request through a layer of 256 fine-grained experts
        dict(name="layer_token", op="layer", tokens=1, experts=256, top_k=8, width=2048, hidden=768, act="silu",
             gated=True, bias=False, residual=True, weights="bf16", logits="fp32", masked=False),
        # 8 requests decoding, weights in MXFP8
        dict(name="layer_batch", op="layer", tokens=8, experts=256, top_k=8, width=2048, hidden=768, act="silu",
             gated=True, bias=False, residual=True, weights="mx", logits="bf16", masked=False),
        # 64 tokens (drafted ones among them, some padding): most of 128 experts are read
        dict(name="layer_full", op="layer", tokens=64, experts=128, top_k=4, width=4096, hidden=1024, act="silu",
             gated=True, bias=False, residual=True, weights="bf16", logits="fp32", masked=True),
        # odd sizes, biases, no gate
        dict(name="layer_odd", op="layer", tokens=5, experts=13, top_k=3, width=1111, hidden=333, act="gelu",
             gated=False, bias=True, residual=False, weights="bf16", logits="fp32", masked=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """Model widths are mostly multiples of 64."""
    n = _log(rng, lo, hi)
    return (n + 63) // 64 * 64 if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_mx", "layer"])
    act, gated = rng.choice(["none", "relu", "gelu", "silu"]), rng.random() < 0.4
    if op == "layer":
        e = _log(rng, 4, 256)
        c = dict(op=op, tokens=_log(rng, 1, 64), experts=e, top_k=rng.randint(1, min(8, e)), width=_size(rng, 256, 5120),
                 hidden=_size(rng, 128, 2048), act=act, gated=gated, bias=rng.random() < 0.3,
                 residual=rng.random() < 0.6, weights=rng.choice(["bf16", "mx"]), logits=rng.choice(["bf16", "fp32"]),
                 masked=rng.random() < 0.3)
        while c["experts"] * c["width"] * c["hidden"] > 128 * 4096 * 1024:
            c["width"], c["hidden"] = c["width"] * 3 // 4, c["hidden"] * 3 // 4
        if c["weights"] == "mx":
            c["width"], c["hidden"] = (c["width"] + 31) // 32 * 32, (c["hidden"] + 31) // 32 * 32
        return c
    c = dict(op=op, rows=_log(rng, 1, 32768), experts=1 if rng.random() < 0.3 else _log(rng, 2, 64),
             width=_size(rng, 64, 8192), out=_size(rng, 64, 8192), act=act, gated=gated, bias=rng.random() < 0.5,
             residual=rng.random() < 0.4, skew=rng.choice([0.0, 0.3, 1.0]))
    if op == "linear":
        c["grad"] = rng.random() < 0.6
    while c["rows"] * c["width"] * c["out"] * (2 if gated else 1) > 1.0e11 or \
            c["experts"] * c["width"] * c["out"] * (2 if gated else 1) > 4.0e8:
        c["width"], c["out"] = c["width"] * 3 // 4, c["out"] * 3 // 4
    if op == "linear_mx":
        c["width"] = (c["width"] + 31) // 32 * 32
    return c


# ---------------------------------------------------------------- inputs

def _group_sizes(case, seed):
    """Rows of each group: a router's choice with more and less popular
    experts; with more than one expert some rows behind the last group stay
    unused."""
    rows, e = case["rows"], case["experts"]
    if e == 1:
        return [rows]
    g = torch.Generator().manual_seed(seed)
    used = rows - int(torch.randint(0, rows // 32 + 1, (1,), generator=g))
    p = torch.softmax(case["skew"] * torch.randn(e, generator=g), 0)
    return torch.bincount(torch.multinomial(p, used, replacement=True, generator=g), minlength=e).tolist()


def _to_mx(x):
    """(q, scales): e4m3 values and biased exponents of blocks of 32."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    code = torch.where(amax > 0, torch.floor(torch.log2(amax)) - 8 + 127, 0.0).clamp(0, 254)
    q = (b * torch.exp2(127.0 - code)).clamp(-448, 448).flatten(-2).to(torch.float8_e4m3fn)
    return q, code[..., 0].to(torch.uint8)


def _weights(e, n, k, g, mx=False):
    w = (torch.randn(e, n, k, generator=g, device="cuda") * k ** -0.5).to(BF16)
    if not mx:
        return w
    parts = [_to_mx(m) for m in w]
    return torch.stack([_codes(p[0]) for p in parts]).view(torch.float8_e4m3fn), torch.stack([p[1] for p in parts])


def _prepare_layer(case, g):
    t, e, d, h = case["tokens"], case["experts"], case["width"], case["hidden"]
    mx = case["weights"] == "mx"
    up_rows = 2 * h if case["gated"] else h
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {"x": new(t, d).to(BF16), "up": _weights(e, up_rows, d, g, mx), "down": _weights(e, d, h, g, mx)}
    logits = 1.5 * new(t, e) + 0.5 * new(1, e)
    s["logits"] = logits.to(BF16 if case["logits"] == "bf16" else torch.float32)
    s["mask"] = torch.rand(t, generator=g, device="cuda") < 0.9 if case["masked"] else None
    s["bias_up"] = 0.1 * new(e, up_rows) if case["bias"] else None
    s["bias_down"] = 0.1 * new(e, d) if case["bias"] else None
    s["residual"] = new(t, d).to(BF16) if case["residual"] else None
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "layer":
        return {"case": case, **_prepare_layer(case, g)}
    r, e, k, n = case["rows"], case["experts"], case["width"], case["out"]
    wide = 2 * n if case["gated"] else n
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    sizes = _group_sizes(case, seed)
    offs = torch.tensor(sizes).cumsum(0).to(torch.int32)
    s = {"case": case, "offs": offs.cuda() if e > 1 else None, "longest": max(sizes), "sizes": sizes}
    x = new(r, k).to(BF16)
    mx = case["op"] == "linear_mx"
    s["x"], s["w"] = _to_mx(x) if mx else x, _weights(e, wide, k, g, mx)
    s["bias"] = 0.1 * new(e, wide) if case["bias"] else None
    s["residual"] = new(r, n).to(BF16) if case["residual"] else None
    if case.get("grad"):
        s["grad_y"] = (1e-2 * new(r, n)).to(BF16)
        # what the forward call saved: unit variance, as the products have
        s["pre"] = new(r, wide).to(BF16) if case["act"] != "none" or case["gated"] else None
    return s


# ---------------------------------------------------------------- plain forms (32 bits)

def _act(x, name):
    if name == "relu":
        return torch.where(x > 0, x, 0.0)
    if name == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _act_slope(x, name):
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if name == "silu":
        sig = 1.0 / (1.0 + torch.exp(-x))
        return sig * (1.0 + x * (1.0 - sig))
    return torch.ones_like(x)


def _full(t):
    """A bf16 tensor, or the values that MXFP8 codes and scales stand for, in 32 bits."""
    if isinstance(t, tuple):
        q, scales = t
        return (q.float().unflatten(-1, (-1, 32)) * torch.exp2(scales.float() - 127.0)[..., None]).flatten(-2)
    return t.float()


def _codes(q):
    return q.view(torch.uint8)


def _padded_rows(s):
    """(E, longest) row numbers, those past a group's end at `rows`, which is no row; and each row's group."""
    r, e = s["case"]["rows"], s["case"]["experts"]
    at = torch.arange(r, device="cuda")
    if e == 1:
        return at[None], torch.zeros_like(at)
    ends = s["offs"].long()
    starts = torch.cat([ends.new_zeros(1), ends[:-1]])
    rows = starts[:, None] + torch.arange(s["longest"], device="cuda")
    return torch.where(rows < ends[:, None], rows, r), torch.searchsorted(ends, at, right=True)


def _gather(x, rows):
    return torch.cat([x, x.new_zeros(1, x.shape[1])])[rows] if rows.shape[0] > 1 else x[None]


def _scatter(y, rows, n):
    """(E, longest, W) back to (n, W); rows of no group are zeros."""
    if rows.shape[0] == 1:
        return y[0]
    out = y.new_zeros(n + 1, y.shape[2])
    out[rows.reshape(-1)] = y.reshape(-1, y.shape[2])
    return out[:n]


def _plain_linear(s):
    c = s["case"]
    n, name, r = c["out"], c["act"], c["rows"]
    rows, group = _padded_rows(s)
    used = (group < c["experts"])[:, None]
    xs, w = _gather(_full(s["x"]), rows), _full(s["w"])
    pre = torch.bmm(xs, w.transpose(1, 2).contiguous())
    if s["bias"] is not None:
        pre = pre + s["bias"][:, None, :]
    y = _act(pre[..., :n], name) * pre[..., n:] if c["gated"] else _act(pre, name)
    y = _scatter(y, rows, r)
    if s["residual"] is not None:
        y = torch.where(used, y + s["residual"].float(), 0.0)
    out = {"y": y.to(BF16)}
    if not c.get("grad"):
        return out
    dy = torch.where(used, s["grad_y"].float(), 0.0)
    if s["pre"] is not None:
        out["pre"] = _scatter(pre, rows, r).to(BF16)
        p = s["pre"].float()
        if c["gated"]:
            gate, value = p[:, :n], p[:, n:]
            dy = torch.cat([dy * value * _act_slope(gate, name), dy * _act(gate, name)], 1)
        else:
            dy = dy * _act_slope(p, name)
    ds = _gather(dy, rows)
    out["grad_x"] = _scatter(torch.bmm(ds, w), rows, r).to(BF16)
    out["grad_w"] = torch.bmm(ds.transpose(1, 2).contiguous(), xs).to(BF16)
    if s["bias"] is not None:
        out["grad_bias"] = ds.sum(1)
    return out


def _plain_layer(s):
    c = s["case"]
    t, k, h, e = c["tokens"], c["top_k"], c["hidden"], c["experts"]
    x, logits = s["x"].float(), s["logits"].float()
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    w = torch.exp(best[:, :k] - best[:, :1])
    w, ids = w / w.sum(1, keepdim=True), ids[:, :k]
    if s["mask"] is not None:
        w = torch.where(s["mask"][:, None], w, 0.0)
    pick = lambda v, i: (_codes(v[0])[i].view(v[0].dtype), v[1][i]) if isinstance(v, tuple) else v[i]  # noqa: E731
    if t * k <= e:  # the weights of every slot's expert
        flat = ids.reshape(-1)
        pre = (_full(pick(s["up"], flat)) * x.repeat_interleave(k, 0)[:, None, :]).sum(2)
        if s["bias_up"] is not None:
            pre = pre + s["bias_up"][flat]
        a = _act(pre[:, :h], c["act"]) * pre[:, h:] if c["gated"] else _act(pre, c["act"])
        z = (_full(pick(s["down"], flat)) * a[:, None, :]).sum(2)
        if s["bias_down"] is not None:
            z = z + s["bias_down"][flat]
        y = (z.view(t, k, -1) * w[:, :, None]).sum(1)
    else:  # every expert on every token
        share = torch.zeros(t, e, device=x.device).scatter_(1, ids, w)
        up = _full(s["up"])
        pre = torch.matmul(x, up.reshape(-1, up.shape[2]).t()).view(t, e, -1)
        if s["bias_up"] is not None:
            pre = pre + s["bias_up"]
        a = _act(pre[..., :h], c["act"]) * pre[..., h:] if c["gated"] else _act(pre, c["act"])
        down = _full(s["down"])
        z = torch.bmm((a * share[:, :, None]).transpose(0, 1).contiguous(), down.transpose(1, 2).contiguous())
        y = z.sum(0)
        if s["bias_down"] is not None:
            y = y + share @ s["bias_down"]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(BF16)}


# ---------------------------------------------------------------- the package's operators

def _run_own(s):
    import mxfp8_quantization_moe_amd as mxq

    c = s["case"]
    if c["op"] == "layer":
        return {"y": mxq.moe_layer(s["x"], s["logits"], s["up"], s["down"], c["top_k"], activation=c["act"],
                                   gated=c["gated"], bias_up=s["bias_up"], bias_down=s["bias_down"],
                                   token_mask=s["mask"], residual=s["residual"])}
    epilogue = dict(bias=s["bias"], activation=c["act"], gated=c["gated"], residual=s["residual"])
    if c["op"] == "linear_mx":
        return {"y": mxq.moe_linear_mx(*s["x"], *s["w"], s["offs"], **epilogue)}
    if not c["grad"]:
        return {"y": mxq.moe_linear(s["x"], s["w"], s["offs"], **epilogue)}
    out = {}
    if s["pre"] is not None:
        out["y"], out["pre"] = mxq.moe_linear(s["x"], s["w"], s["offs"], save_pre=True, **epilogue)
    else:
        out["y"] = mxq.moe_linear(s["x"], s["w"], s["offs"], **epilogue)
    out["grad_x"], out["grad_w"], grad_bias = mxq.moe_linear_backward(
        s["grad_y"], s["x"], s["w"], s["offs"], pre=s["pre"], activation=c["act"], gated=c["gated"], bias=c["bias"])
    if c["bias"]:
        out["grad_bias"] = grad_bias
    return out


def run(state):
    return _run_own(state) if own else (_plain_layer if state["case"]["op"] == "layer" else _plain_linear)(state)


# ---------------------------------------------------------------- work

def work(case):
    wide = 2 if case["gated"] else 1
    if case["op"] == "layer":
        # every expert that some token takes is read once
        t, k, e, d, h = (case[n] for n in ("tokens", "top_k", "experts", "width", "hidden"))
        active = e * (1.0 - (1.0 - k / e) ** t)
        size = 2.0 if case["weights"] == "bf16" else 33.0 / 32.0
        nbytes = active * (wide + 1) * d * h * size + t * d * (6 if case["residual"] else 4) + t * e * 2
        return {"bytes": nbytes, "flops": 2.0 * t * k * d * h * (wide + 1)}
    r, e, k, n = (case[x] for x in ("rows", "experts", "width", "out"))
    size = 2.0 if case["op"] == "linear" else 33.0 / 32.0
    weights = min(e, r) * n * wide * k
    nbytes = r * k * size + weights * size + r * n * (4 if case["residual"] else 2)
    flops = 2.0 * r * n * wide * k
    if case.get("grad"):
        saved = case["act"] != "none" or case["gated"]
        nbytes += (r * n * wide * 4 if saved else 0) + r * n * 2 + r * k * 2 + e * n * wide * k * 2
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_values(t):
    if isinstance(t, tuple):
        return t[0].double() * torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), t[1].int() - 127).repeat_interleave(32, -1)
    return t.double()


def _exact_act(x, name):
    """The activation and its derivative."""
    if name == "none":
        return x, torch.ones_like(x)
    if name == "relu":
        return x.clamp(min=0), (x > 0).double()
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-x / math.sqrt(2.0))
        return x * cdf, cdf + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    sig = torch.sigmoid(x)
    return x * sig, sig + x * sig * (1 - sig)


def _exact_linear(s):
    c = s["case"]
    r, e, n, k, gated = c["rows"], c["experts"], c["out"], c["width"], c["gated"]
    f64 = dict(dtype=torch.float64, device="cuda")
    y = torch.zeros(r, n, **f64)
    out = {"y": y}
    if c.get("grad"):
        wide = 2 * n if gated else n
        if s["pre"] is not None:
            out["pre"] = torch.zeros(r, wide, **f64)
        out["grad_x"] = torch.zeros(r, k, **f64)
        out["grad_w"] = torch.zeros(e, wide, k, **f64)
        if s["bias"] is not None:
            out["grad_bias"] = torch.zeros(e, wide, **f64)
    lo = 0
    for i, size in enumerate(s["sizes"]):
        at, lo = slice(lo, lo + size), lo + size
        if not size:
            continue
        x = _exact_values((s["x"][0][at], s["x"][1][at]) if isinstance(s["x"], tuple) else s["x"][at])
        w = _exact_values((s["w"][0][i], s["w"][1][i]) if isinstance(s["w"], tuple) else s["w"][i])
        z = x @ w.t()
        if s["bias"] is not None:
            z += s["bias"][i].double()
        y[at] = _exact_act(z[:, :n], c["act"])[0] * (z[:, n:] if gated else 1.0)
        if s["residual"] is not None:
            y[at] += s["residual"][at].double()
        if not c.get("grad"):
            continue
        dz = s["grad_y"][at].double()
        if s["pre"] is not None:
            out["pre"][at] = z
            p = s["pre"][at].double()
            a, slope = _exact_act(p[:, :n], c["act"])
            dz = torch.cat([dz * p[:, n:] * slope, dz * a], 1) if gated else dz * slope
        out["grad_x"][at] = dz @ w
        out["grad_w"][i] = dz.t() @ x
        if s["bias"] is not None:
            out["grad_bias"][i] = dz.sum(0)
    return out


def _exact_layer(s):
    c = s["case"]
    h, k = c["hidden"], c["top_k"]
    logits, x = s["logits"].double(), s["x"].double()
    y = s["residual"].double() if s["residual"] is not None else torch.zeros_like(x)
    rows = logits.cpu().tolist()
    ids = [sorted(range(c["experts"]), key=lambda e: (-row[e], e))[:k] for row in rows]  # noqa: B023
    for e in sorted(set(sum(ids, []))):
        tokens = [t for t in range(c["tokens"]) if e in ids[t] and (s["mask"] is None or bool(s["mask"][t]))]
        if not tokens:
            continue
        up, down = (_exact_values((m[0][e], m[1][e]) if isinstance(m, tuple) else m[e]) for m in (s["up"], s["down"]))
        z = x[tokens] @ up.t()
        if s["bias_up"] is not None:
            z = z + s["bias_up"][e].double()
        a = _exact_act(z[:, :h], c["act"])[0] * (z[:, h:] if c["gated"] else 1.0)
        z = a @ down.t()
        if s["bias_down"] is not None:
            z = z + s["bias_down"][e].double()
        share = [math.exp(rows[t][e]) / sum(math.exp(rows[t][i]) for i in ids[t]) for t in tokens]
        y[tokens] += z * torch.tensor(share, dtype=torch.float64, device="cuda")[:, None]
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_layer(s) if case["op"] == "layer" else _exact_linear(s)

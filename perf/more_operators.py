"""Cases of the operators around the expert layer, with their plain forms.

- ``balance``: how evenly a batch's routing loads the experts: pairs per sequence and expert, the
  balance loss of the router's normalised scores, and the gradient of the router's logits from that
  loss and from the applied weights;
- ``norm``: the step between two blocks of the residual stream, out = a x + b gate * norm(y) and the
  next block's norm of it, alone or with its gradients;
- ``adapter``: low-rank adapters of many requests beside one projection they share,
  y = base + s (x A^T) B^T with each request's own A, B and s.

``own = False`` computes them from elementary torch operations in 32 bits; ``own = True``
calls the library.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-5
# the type of a logit's gradient: a token's part of a batch's loss lies below fp16's normal numbers
_GRAD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float32}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # counts and loss of a small padded batch while a router is watched, no gradient
        {"name": "balance small", "op": "balance", "T": 64, "E": 64, "top": 4, "S": 3, "varied": True, "masked": True,
         "train": False, "weights": False, "type": "bf16"},
        # a training step's router over a batch of sequences, 256 experts
        {"name": "balance batch", "op": "balance", "T": 4096, "E": 256, "top": 8, "S": 4, "varied": False, "masked": False,
         "train": True, "weights": True, "type": "f32"},
        # odd sizes: ragged padded sequences, a number of experts off every grid
        {"name": "balance odd", "op": "balance", "T": 5003, "E": 333, "top": 7, "S": 29, "varied": True, "masked": True,
         "train": True, "weights": True, "type": "f16"},
        # a large batch over a wide layer
        {"name": "balance large", "op": "balance", "T": 65536, "E": 384, "top": 8, "S": 16, "varied": False, "masked": False,
         "train": True, "weights": True, "type": "f32"},
        # one token between two blocks of a served model: pure latency
        {"name": "norm one token", "op": "norm", "T": 1, "H": 6144, "post": True, "gate": "none", "pre": True,
         "train": False, "stream": "bf16", "type": "bf16"},
        # a decode batch on an fp32 stream, a shared expert's gate a token
        {"name": "norm decode", "op": "norm", "T": 64, "H": 7168, "post": False, "gate": "token", "pre": True,
         "train": False, "stream": "f32", "type": "bf16"},
        # a training step on odd sizes, a learned scale a channel
        {"name": "norm train odd", "op": "norm", "T": 333, "H": 1000, "post": True, "gate": "channel", "pre": True,
         "train": True, "stream": "f32", "type": "f16"},
        # a training step between two blocks of a large model, every element with its gate
        {"name": "norm train", "op": "norm", "T": 8192, "H": 6144, "post": True, "gate": "full", "pre": True,
         "train": True, "stream": "bf16", "type": "bf16"},
        # one token with one adapter beside a down projection: pure latency
        {"name": "adapter one token", "op": "adapter", "T": 1, "S": 1, "K": 2048, "N": 6144, "rank": 16, "A": 4,
         "free": 0.0, "type": "bf16", "out": "bf16"},
        # a decode batch: 64 requests, 32 adapters, some requests without one
        {"name": "adapter decode", "op": "adapter", "T": 64, "S": 64, "K": 6144, "N": 2048, "rank": 16, "A": 32,
         "free": 0.2, "type": "bf16", "out": "f32"},
        # a few short prompts on odd sizes
        {"name": "adapter odd", "op": "adapter", "T": 777, "S": 11, "K": 1000, "N": 520, "rank": 24, "A": 7,
         "free": 0.2, "type": "f16", "out": "f16"},
        # prompts of several requests through a square projection
        {"name": "adapter prompts", "op": "adapter", "T": 8192, "S": 6, "K": 6144, "N": 6144, "rank": 64, "A": 6,
         "free": 0.0, "type": "bf16", "out": "bf16"},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, evenly over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["balance", "norm", "adapter"])
    if op == "balance":
        e = _spread(rng, 8, 384)
        t = _spread(rng, 1, 40000)
        return {"op": op, "T": t, "E": e, "top": rng.randint(1, min(e, 12)), "S": min(t, _spread(rng, 1, 60)),
                "varied": rng.random() < 0.5, "masked": rng.random() < 0.4, "train": rng.random() < 0.7,
                "weights": rng.random() < 0.6, "type": rng.choice(["f32", "bf16", "f16"])}
    if op == "norm":
        return {"op": op, "T": _spread(rng, 1, 6000), "H": _spread(rng, 64, 7168, 8), "post": rng.random() < 0.5,
                "gate": rng.choice(["none", "channel", "token", "full"]), "pre": rng.random() < 0.8,
                "train": rng.random() < 0.5, "stream": rng.choice(["f32", "bf16"]),
                "type": rng.choice(["f32", "bf16", "f16"])}
    t = _spread(rng, 1, 6000)
    s = t if t <= 100 and rng.random() < 0.6 else min(t, _spread(rng, 1, 16))
    return {"op": op, "T": t, "S": s, "K": _spread(rng, 256, 6144, 8), "N": _spread(rng, 256, 6144, 8),
            "rank": rng.choice([8, 16, 24, 32, 64]), "A": rng.choice([1, 5, 16, 32]), "free": rng.choice([0.0, 0.3]),
            "type": rng.choice(["bf16", "f16"]), "out": rng.choice(["bf16", "f16", "f32"])}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _cuts(g, t, s):
    """s lengths of a ragged batch of t rows (one each where s = t), and their offsets on the GPU."""
    if s == t:
        ends = torch.arange(t + 1)
    else:
        inner = torch.sort(torch.randint(0, t + 1, (s - 1,), generator=g, device="cuda"))[0].cpu()
        ends = torch.cat([torch.zeros(1, dtype=torch.long), inner, torch.full((1,), t)])
    return (ends[1:] - ends[:-1]).tolist(), ends.to(device="cuda", dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _TYPES[case["type"]]
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    rand = lambda *n: torch.rand(*n, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "balance":
        t, e, k = case["T"], case["E"], case["top"]
        s["lengths"], s["offsets"] = _cuts(g, t, case["S"])
        logits = (1.2 * randn(t, e) + 0.5 * randn(e)).to(dt)      # some experts are liked more than others
        s["logits"] = logits
        # chosen by score and selection bias, as the router does
        s["ids"] = (torch.sigmoid(logits.float()) + 0.1 * randn(e)).topk(k, dim=1)[1].to(torch.int32)
        s["keff"] = torch.full((t,), k, dtype=torch.int32, device="cuda")
        if case["varied"]:
            s["keff"] = torch.randint(1, k + 1, (t,), generator=g, device="cuda", dtype=torch.int32)
            s["ids"][torch.arange(k, device="cuda")[None] >= s["keff"][:, None]] = -1
        s["valid"] = (rand(t) >= 0.1).to(torch.uint8) if case["masked"] else None
        s["dloss"] = torch.tensor([0.01], device="cuda")
        s["dw"] = randn(t, k) / t if case["weights"] else None
        s["scale"] = 2.5
    elif case["op"] == "norm":
        t, h = case["T"], case["H"]
        st = _TYPES[case["stream"]]
        s["x"] = (randn(t, h) * torch.exp(0.5 * randn(t, 1))).to(st)
        s["y"] = (0.5 * randn(t, h)).to(dt)
        s["post"] = 1 + 0.1 * randn(h) if case["post"] else None
        s["pre"] = 1 + 0.1 * randn(h) if case["pre"] else None
        shape = {"none": None, "channel": (1, h), "token": (t, 1), "full": (t, h)}[case["gate"]]
        s["gate"] = (0.5 + 0.5 * randn(*shape)).to(dt) if shape else None
        s["a"], s["b"] = 1.0, 0.75
        if case["train"]:
            s["dout"] = randn(t, h).to(st)
            s["dn"] = randn(t, h).to(dt) if case["pre"] else None
    else:
        t, k, n, r, a = case["T"], case["K"], case["N"], case["rank"], case["A"]
        s["lengths"], s["offsets"] = _cuts(g, t, case["S"])
        ids = torch.randint(0, a, (case["S"],), generator=g, device="cuda", dtype=torch.int32)
        ids[rand(case["S"]) < case["free"]] = -1
        s["ids"], s["host_ids"] = ids, ids.tolist()
        s["x"] = randn(t, k).to(dt)
        s["down"] = (randn(a, r, k) / math.sqrt(k)).to(dt)
        s["up"] = (0.5 * randn(a, n, r) / math.sqrt(r)).to(dt)
        s["scale"] = 0.5 + 1.5 * rand(a)
        s["base"] = randn(t, n).to(_TYPES[case["out"]])
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------
def _plain_balance(s):
    c = s["case"]
    t, e, k, n = c["T"], c["E"], c["top"], c["S"]
    sig = 1.0 / (1.0 + torch.exp(-s["logits"].float()))
    total = sig.sum(1, keepdim=True)
    p = sig / total
    at = torch.arange(t, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"], at, right=True) - 1
    counted = torch.ones(t, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"] != 0
    of_seq = ((torch.arange(n, device="cuda")[:, None] == seq[None]) & counted[None]).float()      # [S][T]
    tokens = of_seq.sum(1)
    kept = (torch.arange(k, device="cuda")[None] < s["keff"][:, None]) & counted[:, None]
    ids = torch.where(kept, s["ids"].long(), e)
    counts = torch.zeros(n * (e + 1), dtype=torch.int32, device="cuda")
    counts.index_add_(0, (seq[:, None] * (e + 1) + ids).reshape(-1), torch.ones(t * k, dtype=torch.int32, device="cuda"))
    counts = counts.view(n, e + 1)[:, :e].contiguous()
    load = counts.float() * (e / counts.sum(1, keepdim=True).clamp_min(1).float())
    used = (tokens > 0).float()
    each = used / (tokens.clamp_min(1) * used.sum().clamp_min(1))        # a token's share of the loss
    loss = (load * torch.matmul(of_seq, p) * each[:, None]).sum()
    out = {"loss": loss, "counts": counts}
    if not c["train"]:
        return out
    grad = (load * each[:, None])[seq] * s["dloss"]
    ds = (grad - (grad * p).sum(1, keepdim=True)) / total
    if s["dw"] is not None:
        kept_sig = torch.where(kept, torch.gather(sig, 1, ids.clamp_max(e - 1)), torch.zeros(1, device="cuda"))
        dw = torch.where(kept, s["dw"], torch.zeros(1, device="cuda"))
        norm = kept_sig.sum(1, keepdim=True)
        norm = torch.where(norm > 0, norm, torch.ones_like(norm))
        dg = torch.where(kept, s["scale"] / norm * (dw - (dw * kept_sig).sum(1, keepdim=True) / norm), torch.zeros(1, device="cuda"))
        ds = ds + torch.zeros(t, e + 1, device="cuda").scatter_add_(1, ids, dg)[:, :e]
    out["dlogits"] = torch.where(counted[:, None], ds * sig * (1.0 - sig), torch.zeros(1, device="cuda")).to(_GRAD[c["type"]])
    return out


def _inverse(v):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + _EPS)


def _plain_norm(s):
    c = s["case"]
    st, dt = _TYPES[c["stream"]], _TYPES[c["type"]]
    x, y = s["x"].float(), s["y"].float()
    gate = s["gate"].float() if s["gate"] is not None else None
    z, iy = y, None
    if s["post"] is not None:
        iy = _inverse(y)
        z = y * iy * s["post"]
    out = s["a"] * x + s["b"] * (z if gate is None else gate * z)
    r = {"out": out.to(st)}
    if s["pre"] is not None:
        io = _inverse(out)
        r["n"] = (out * io * s["pre"]).to(dt)
    if not c["train"]:
        return r
    d = s["dout"].float()
    if s["pre"] is not None:
        dn = s["dn"].float()
        w = dn * s["pre"]
        d = d + io * (w - out * (io * io * (w * out).mean(1, keepdim=True)))
        r["dpre"] = (dn * out * io).sum(0)
    r["dx"] = (s["a"] * d).to(st)
    dz = s["b"] * (d if gate is None else d * gate)
    if gate is not None:
        dgate = s["b"] * d * z
        if c["gate"] == "channel":
            dgate = dgate.sum(0, keepdim=True)
        if c["gate"] == "token":
            dgate = dgate.sum(1, keepdim=True)
        r["dgate"] = dgate.to(dt) if c["gate"] == "full" else dgate
    if s["post"] is not None:
        w = dz * s["post"]
        r["dpost"] = (dz * y * iy).sum(0)
        dz = iy * (w - y * (iy * iy * (w * y).mean(1, keepdim=True)))
    r["dy"] = dz.to(dt)
    return r


def _plain_adapter(s):
    y = s["base"].float()
    at = 0
    parts = []
    for length, a in zip(s["lengths"], s["host_ids"]):
        rows = y[at:at + length]
        if a >= 0 and length:
            u = torch.matmul(s["x"][at:at + length].float(), s["down"][a].float().t())
            rows = rows + s["scale"][a] * torch.matmul(u, s["up"][a].float().t())
        parts.append(rows)
        at += length
    return torch.cat(parts).to(_TYPES[s["case"]["out"]])


# ---------------------------------------------------------------------------------------
# the library
# ---------------------------------------------------------------------------------------
def _buffers(s, moe):
    """The outputs and the workspace that a program keeps from call to call."""
    c = s["case"]
    empty = lambda *shape, t: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
    f32, i32 = torch.float32, torch.int32
    if c["op"] == "balance":
        cfg = moe.MoeConfig.make(64, c["E"], c["top"], 64, routed_scaling_factor=s["scale"])
        return {"cfg": cfg, "loss": empty(1, t=f32), "counts": empty(c["S"], c["E"], t=i32), "tokens": empty(c["S"], t=i32),
                "dlogits": torch.empty_like(s["logits"], dtype=_GRAD[c["type"]]), "workspace": moe.alloc_balance_workspace(cfg, c["T"], c["S"])}
    if c["op"] == "norm":
        t, h = c["T"], c["H"]
        b = {"out": torch.empty_like(s["x"]), "n": torch.empty_like(s["y"]) if c["pre"] else None}
        if c["train"]:
            b |= {"kept": empty(t, 2, t=f32), "dx": torch.empty_like(s["x"]), "dy": torch.empty_like(s["y"]),
                  "dpre": empty(h, t=f32) if c["pre"] else None, "dpost": empty(h, t=f32) if c["post"] else None,
                  "dgate": None, "workspace": moe.alloc_block_norm_workspace(t, h)}
            if s["gate"] is not None:
                b["dgate"] = empty(*s["gate"].shape, t=_TYPES[c["type"]] if c["gate"] == "full" else f32)
        return b
    return {"y": torch.empty_like(s["base"]), "workspace": moe.alloc_adapter_workspace()}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"balance": _plain_balance, "norm": _plain_norm, "adapter": _plain_adapter}[c["op"]](s)
    import sparse_expert_ffn_route_gb300 as moe
    b = s.get("own") or s.setdefault("own", _buffers(s, moe))
    if c["op"] == "balance":
        moe.moe_balance_forward(b["cfg"], s["logits"], s["ids"], s["keff"], s["offsets"], b["loss"], b["counts"], b["tokens"],
                                b["workspace"], valid=s["valid"])
        out = {"loss": b["loss"][0], "counts": b["counts"]}
        if c["train"]:
            moe.moe_balance_backward(b["cfg"], s["logits"], s["ids"], s["keff"], s["offsets"], b["counts"], b["tokens"],
                                     b["dlogits"], b["workspace"], dloss=s["dloss"], dw=s["dw"], valid=s["valid"])
            out["dlogits"] = b["dlogits"]
        return out
    if c["op"] == "norm":
        moe.moe_block_norm_forward(s["x"], _EPS, y=s["y"], post_w=s["post"], gate=s["gate"], pre_w=s["pre"], out=b["out"],
                                   n=b["n"], residual_scale=s["a"], branch_scale=s["b"], kept=b.get("kept"))
        out = {"out": b["out"]} | ({"n": b["n"]} if c["pre"] else {})
        if c["train"]:
            moe.moe_block_norm_backward(s["x"], b["kept"], b["workspace"], y=s["y"], post_w=s["post"], gate=s["gate"],
                                        pre_w=s["pre"], dout=s["dout"], dn=s["dn"], dx=b["dx"], dy=b["dy"], dgate=b["dgate"],
                                        dpost=b["dpost"], dpre=b["dpre"], residual_scale=s["a"], branch_scale=s["b"])
            out |= {k: b[k] for k in ("dpre", "dx", "dgate", "dpost", "dy") if b[k] is not None}
        return out
    moe.moe_adapter_matmul(s["x"], s["down"], s["up"], s["scale"], s["offsets"], s["ids"], b["y"], b["workspace"],
                           base=s["base"])
    return b["y"]


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    b = _BYTES[case["type"]]
    if case["op"] == "balance":
        t, e, k = case["T"], case["E"], case["top"]
        n = b * t * e + 4 * t * (k + 1) + 4 * case["S"] * e
        if case["train"]:       # the logits are read once for both
            n += (2 if case["type"] == "bf16" else 4) * t * e + (4 * t * k if case["weights"] else 0)
        return {"bytes": n, "flops": (8 if case["train"] else 4) * t * e}
    if case["op"] == "norm":
        t, h, r = case["T"], case["H"], _BYTES[case["stream"]]
        gate = {"none": 0, "channel": h, "token": t, "full": t * h}[case["gate"]]
        n = t * h * (2 * r + b * (1 + case["pre"])) + b * gate + 4 * h * (case["post"] + case["pre"])
        if case["train"]:       # dout and dn in, dx, dy, the gate's and the weights' gradients out
            n += t * h * (2 * r + b * (1 + case["pre"])) + (b if case["gate"] == "full" else 4) * gate
            n += 4 * h * (case["post"] + case["pre"])
        return {"bytes": n, "flops": (30 if case["train"] else 10) * t * h}
    t, k, n, r = case["T"], case["K"], case["N"], case["rank"]
    busy = max(1.0, case["S"] * (1 - case["free"]))
    used = case["A"] * (1 - (1 - 1 / case["A"]) ** busy)      # distinct adapters of an even choice
    part = 1 - case["free"]
    return {"bytes": b * (part * t * k + used * r * (k + n)) + 2 * _BYTES[case["out"]] * t * n,
            "flops": 2 * part * t * r * (k + n)}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_balance(case, s):
    e = case["E"]
    scores = torch.sigmoid(s["logits"].double())
    share = scores / scores.sum(1, keepdim=True)
    valid = torch.ones(case["T"], device="cuda") if s["valid"] is None else s["valid"]
    hot = torch.zeros(case["T"], e, dtype=torch.float64, device="cuda")      # pairs of (token, expert)
    for i in range(case["top"]):
        rows = ((s["keff"] > i) & (valid != 0)).nonzero()[:, 0]
        hot[rows, s["ids"][rows, i].long()] += 1
    pieces = [slice(a, a + n) for a, n in zip(s["offsets"].tolist(), s["lengths"])]
    filled = [bool(n) and bool(valid[p].any()) for p, n in zip(pieces, s["lengths"])]
    counts = torch.stack([hot[p].sum(0) for p in pieces])
    loss = 0.0
    d = torch.zeros_like(scores)
    for p, f, cnt in zip(pieces, filled, counts):
        if not f:
            continue
        v = valid[p].double()[:, None]
        slope = cnt * e / cnt.sum().clamp_min(1) / v.sum() / sum(filled)
        loss = loss + (v * share[p] * slope).sum()
        d[p] = v * float(s["dloss"]) * (slope - share[p] @ slope[:, None]) / scores[p].sum(1, keepdim=True)
    out = {"loss": torch.as_tensor(loss, dtype=torch.float64, device="cuda"), "counts": counts}
    if not case["train"]:
        return out
    if s["dw"] is not None:
        # w = scale * g / sum(g) over the kept ones, by the quotient rule
        g = hot * scores
        total = g.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        dw = torch.zeros_like(d)
        for i in range(case["top"]):
            rows = ((s["keff"] > i) & (valid != 0)).nonzero()[:, 0]
            dw[rows, s["ids"][rows, i].long()] = s["dw"][rows, i].double()
        d += s["scale"] * hot * (dw / total - (dw * g).sum(1, keepdim=True) / total ** 2)
    out["dlogits"] = d * scores * (1 - scores)
    return out


def _exact_norm(case, s):
    """Forward and, by the chain rule on unit vectors of the norms, backward."""
    x, y = s["x"].double(), s["y"].double()
    h = x.shape[1]
    gate = torch.ones(1, 1, dtype=torch.float64, device="cuda") if s["gate"] is None else s["gate"].double()
    size = lambda v: torch.sqrt(v.square().sum(1, keepdim=True) / h + _EPS)  # noqa: E731
    unit = y / size(y)
    z = unit * s["post"].double() if case["post"] else y
    out = x * s["a"] + z * gate * s["b"]
    r = {"out": out}
    if case["pre"]:
        unit_out = out / size(out)
        r["n"] = unit_out * s["pre"].double()
    if not case["train"]:
        return r

    def through(du, u, v):      # d/dv of v / size(v), u = v / size(v)
        return (du - u * (du * u).sum(1, keepdim=True) / h) / size(v)
    d = s["dout"].double()
    if case["pre"]:
        r["dpre"] = torch.einsum("th,th->h", s["dn"].double(), unit_out)
        d = d + through(s["dn"].double() * s["pre"].double(), unit_out, out)
    r["dx"] = d * s["a"]
    if case["gate"] != "none":
        over = {"channel": 0, "token": 1}.get(case["gate"])
        r["dgate"] = d * z * s["b"] if over is None else (d * z).sum(over, keepdim=True) * s["b"]
    dz = d * gate * s["b"]
    if case["post"]:
        r["dpost"] = torch.einsum("th,th->h", dz, unit)
        dz = through(dz * s["post"].double(), unit, y)
    r["dy"] = dz
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(case, s)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    y = s["base"].double()
    ends = s["offsets"].tolist()
    for i, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            p = slice(ends[i], ends[i + 1])
            y[p] += (s["x"][p].double() @ s["down"][a].double().T) @ s["up"][a].double().T * float(s["scale"][a])
    return y

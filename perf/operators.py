"""Cases of the MXFP4 and gated feed-forward operators, with their plain forms.

Four operators of the feed-forward part of a mixture-of-experts decoder:

- ``quantize``: rows to MXFP4 (4-bit e2m1 codes, one power-of-two scale for 32 values) and
  back to the values that the codes stand for;
- ``product``: the product of MXFP4 rows with MXFP4 weights, grouped by expert;
- ``experts``: the expert feed-forward block on MXFP4 weights, from the tokens and their
  grouping by expert to one output row for each (token, expert) pair;
- ``gated``: the dense gated block in 16 bits, h = silu(x Wg^T) * (x Wu^T), with its gradients.

``own = False`` computes them from elementary torch operations in 32 bits; ``own = True``
calls the library.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one token's activations before an MXFP4 product: pure latency
        {"name": "quantize one token", "op": "quantize", "rows": 1, "K": 6144, "type": "bf16"},
        # a batch of activations with a ragged width
        {"name": "quantize ragged", "op": "quantize", "rows": 1009, "K": 1120, "type": "f16"},
        # the gate matrices of eight experts, converted from fp32
        {"name": "quantize weights", "op": "quantize", "rows": 16384, "K": 6144, "type": "f32"},
        # one token through a shared expert's down projection
        {"name": "product one token", "op": "product", "rows": 1, "N": 6144, "K": 2048, "E": 1, "type": "bf16"},
        # a few rows over three ragged matrices, the middle of the range in odd sizes
        {"name": "product odd", "op": "product", "rows": 77, "N": 1000, "K": 1120, "E": 3, "type": "f32"},
        # a prompt through a square projection
        {"name": "product prompt", "op": "product", "rows": 4096, "N": 6144, "K": 6144, "E": 1, "type": "bf16"},
        # one token through a small layer's experts
        {"name": "experts one token", "op": "experts", "T": 1, "H": 2048, "F": 512, "E": 256, "top": 8, "skew": 0.0, "type": "bf16"},
        # a decode batch through a large layer's experts: the weights' stream
        {"name": "experts decode", "op": "experts", "T": 32, "H": 6144, "F": 2048, "E": 256, "top": 8, "skew": 0.0, "type": "bf16"},
        # a prompt through the same layer, experts unevenly loaded
        {"name": "experts prompt", "op": "experts", "T": 4096, "H": 6144, "F": 2048, "E": 256, "top": 8, "skew": 0.5, "type": "bf16"},
        # one token through the 16-bit block (no gradient)
        {"name": "gated one token", "op": "gated", "T": 1, "H": 6144, "F": 2048, "train": False, "type": "bf16"},
        # a training step on odd sizes in fp16
        {"name": "gated train odd", "op": "gated", "T": 333, "H": 1000, "F": 520, "train": True, "type": "f16"},
        # a training step of a dense layer
        {"name": "gated train", "op": "gated", "T": 4096, "H": 6144, "F": 2048, "train": True, "type": "bf16"},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, evenly over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = max(lo, min(hi, int(round(v / step)) * step))
    return v + step if v == 3 * 1024 else v


def draw(rng):
    op = rng.choice(["quantize", "product", "experts", "gated"])
    kind = rng.choice(["bf16", "f16", "f32"])
    if op == "quantize":
        return {"op": op, "rows": _spread(rng, 1, 16000), "K": _spread(rng, 32, 6144, 32), "type": kind}
    if op == "product":
        e = rng.choice([1, 1, 2, 5, 8])
        return {"op": op, "rows": _spread(rng, 1, 4000), "N": _spread(rng, 16, 6000), "K": _spread(rng, 32, 6144, 32),
                "E": e, "type": kind}
    if op == "experts":
        return {"op": op, "T": _spread(rng, 1, 4000), "H": _spread(rng, 256, 6144, 64), "F": _spread(rng, 128, 2048, 64),
                "E": rng.choice([8, 32, 64, 128, 256]), "top": rng.choice([2, 4, 8]), "skew": rng.choice([0.0, 0.5]),
                "type": rng.choice(["bf16", "f16"])}
    return {"op": op, "T": _spread(rng, 1, 4000), "H": _spread(rng, 64, 6144, 8), "F": _spread(rng, 64, 2048, 8),
            "train": rng.random() < 0.6, "type": rng.choice(["bf16", "f16"])}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _weights(g, groups, n, k):
    """MXFP4 weights [groups][n][k]: uniform codes, scales around the one that gives
    products of unit size (a uniform code's mean square is 8.6)."""
    codes = torch.randint(0, 256, (groups, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    e = 127 + round(math.log2(1.0 / (2.93 * math.sqrt(k))))
    scales = torch.randint(e - 1, e + 2, (groups, n, k // 32), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _TYPES[case["type"]]
    s = {"case": case}
    if case["op"] == "quantize":
        x = torch.randn(case["rows"], case["K"], generator=g, device="cuda")
        x *= torch.exp(torch.randn(case["rows"], 1, generator=g, device="cuda"))   # rows of differing size
        x[torch.rand(x.shape, generator=g, device="cuda") < 0.01] = 0.0
        s["x"] = x.to(dt)
    elif case["op"] == "product":
        rows, k, e = case["rows"], case["K"], case["E"]
        x, xs = _weights(g, 1, rows, k)
        s["x"], s["xs"] = x[0], xs[0]
        s["w"], s["ws"] = _weights(g, e, case["N"], k)
        cut = torch.sort(torch.randint(0, rows + 1, (e - 1,), generator=g, device="cuda", dtype=torch.int32))[0]
        ends = torch.tensor([0, rows], device="cuda", dtype=torch.int32)
        s["offsets"] = torch.cat([ends[:1], cut, ends[1:]])
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    elif case["op"] == "experts":
        t, h, f, e, top = case["T"], case["H"], case["F"], case["E"], case["top"]
        s["x"] = torch.randn(t, h, generator=g, device="cuda")
        s["wg"], s["wu"], s["wd"] = _weights(g, e, f, h), _weights(g, e, f, h), _weights(g, e, h, f)
        # top experts of each token from skewed logits, then the pairs in expert order
        u = torch.rand(t, e, generator=g, device="cuda").clamp_min(1e-9)
        rank = torch.randperm(e, generator=g, device="cuda") + 1
        ids = (-torch.log(-torch.log(u)) - case["skew"] * torch.log(rank.float())).topk(top, dim=1)[1].reshape(-1)
        order = torch.sort(ids, stable=True)[1]
        s["tok"] = torch.div(order, top, rounding_mode="floor").to(torch.int32)
        counts = torch.bincount(ids, minlength=e)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["uniq"] = counts.nonzero().flatten()
        s["most"] = int(counts.max())
    else:
        t, h, f = case["T"], case["H"], case["F"]
        s["x"] = torch.randn(t, h, generator=g, device="cuda").to(dt)
        s["wg"] = (torch.randn(f, h, generator=g, device="cuda") / math.sqrt(h)).to(dt)
        s["wu"] = (torch.randn(f, h, generator=g, device="cuda") / math.sqrt(h)).to(dt)
        if case["train"]:
            s["dh"] = torch.randn(t, f, generator=g, device="cuda").to(dt)
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------
def _to_codes(x):
    """fp32 rows [.., K] -> magnitude codes 0..7, negative where, exponents [.., K/32]."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 3).clamp(-126, 127)     # floor(log2(amax)) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -126))
    a = torch.ldexp(b.abs(), -e.unsqueeze(-1))
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code, b < 0, e


def _grid(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)


def _round_trip(x):
    code, neg, e = _to_codes(x)
    v = torch.ldexp(_grid(x.device)[code], e.unsqueeze(-1))
    return torch.where(neg, -v, v).reshape(x.shape)


def _values(codes, scales):
    """MXFP4 codes [.., K/2] (low nibble first) and scales [.., K/32] -> fp32 [.., K]."""
    table = torch.cat([_grid(codes.device), -_grid(codes.device)])
    both = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    v = both.reshape(*scales.shape, 32) * torch.exp2(scales.float() - 127.0).unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], -1)


def _by_group(rows, offsets, most):
    """rows [P][..] in group order -> [groups][most][..] (zeros behind a group's end), and
    each row's (group, place)."""
    at = torch.arange(rows.shape[0], device=rows.device, dtype=torch.int32)
    group = (torch.searchsorted(offsets, at, right=True) - 1).long()
    place = at.long() - offsets.long()[group]
    out = rows.new_zeros(offsets.shape[0] - 1, max(most, 1), rows.shape[1])
    out[group, place] = rows
    return out, group, place


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain(s):
    c = s["case"]
    dt = _TYPES[c["type"]]
    if c["op"] == "quantize":
        return _round_trip(s["x"].float()).to(dt)
    if c["op"] == "product":
        x, group, place = _by_group(_values(s["x"], s["xs"]), s["offsets"], s["most"])
        return torch.matmul(x, _values(s["w"], s["ws"]).transpose(1, 2))[group, place].to(dt)
    if c["op"] == "experts":
        of = lambda w: _values(w[0][s["uniq"]], w[1][s["uniq"]]).transpose(1, 2)  # noqa: E731
        offsets = torch.cat([s["offsets"][s["uniq"]], s["offsets"][-1:]])
        x, group, place = _by_group(_round_trip(s["x"])[s["tok"].long()], offsets, s["most"])
        h = torch.matmul(x, of(s["wg"]))
        h = _silu(h) * torch.matmul(x, of(s["wu"]))
        return torch.matmul(_round_trip(h), of(s["wd"]))[group, place].to(dt)
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
    sig = 1.0 / (1.0 + torch.exp(-g))
    h = (g * sig * u).to(dt)
    if not c["train"]:
        return h
    dh = s["dh"].float()
    dg, du = dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig
    return {"h": h, "dx": (torch.matmul(dg, wg) + torch.matmul(du, wu)).to(dt),
            "dw_gate": torch.matmul(dg.t(), x).to(dt), "dw_up": torch.matmul(du.t(), x).to(dt)}


# ---------------------------------------------------------------------------------------
# the library
# ---------------------------------------------------------------------------------------
def _buffers(s, moe):
    """The outputs and the workspace that a program keeps from call to call."""
    c = s["case"]
    dt = _TYPES[c["type"]]
    empty = lambda *shape, t=dt: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
    if c["op"] == "quantize":
        return {"codes": empty(c["rows"], c["K"] // 2, t=torch.uint8), "scales": empty(c["rows"], c["K"] // 32, t=torch.uint8),
                "y": empty(c["rows"], c["K"])}
    if c["op"] == "product":
        return {"y": empty(c["rows"], c["N"]), "workspace": moe.alloc_mxfp4_matmul_workspace()}
    if c["op"] == "experts":
        cfg = moe.MoeConfig.make(c["H"], c["E"], c["top"], c["F"])
        w = {n + "_" + m: s[k][i] for k, m in (("wg", "gate"), ("wu", "up"), ("wd", "down")) for i, n in enumerate("ws")}
        return {"cfg": cfg, "w": w, "y": empty(c["T"] * c["top"], c["H"]), "workspace": moe.alloc_mxfp4_workspace(cfg, c["T"])}
    t, h, f = c["T"], c["H"], c["F"]
    b = {"h": empty(t, f), "workspace": moe.alloc_gated_workspace(t, h, f, c["train"])}
    if c["train"]:
        b |= {"g": empty(t, f), "u": empty(t, f), "dx": empty(t, h), "dwg": empty(f, h), "dwu": empty(f, h)}
    return b


def run(state):
    if not own:
        return _plain(state)
    import sparse_expert_ffn_route_gb300 as moe
    s, c = state, state["case"]
    b = s.get("own") or s.setdefault("own", _buffers(s, moe))
    if c["op"] == "quantize":
        moe.moe_quantize_mxfp4(s["x"], b["codes"], b["scales"])
        moe.moe_dequantize_mxfp4(b["codes"], b["scales"], b["y"])
        return b["y"]
    if c["op"] == "product":
        moe.moe_mxfp4_matmul(s["x"], s["xs"], s["w"], s["ws"], b["y"], b["workspace"], offsets=s["offsets"])
        return b["y"]
    if c["op"] == "experts":
        moe.moe_mxfp4_expert_ffn(b["cfg"], s["x"], b["w"], b["y"], b["workspace"], offsets=s["offsets"], tok=s["tok"])
        return b["y"]
    if not c["train"]:
        moe.moe_gated_forward(s["x"], s["wg"], s["wu"], b["h"], b["workspace"])
        return b["h"]
    moe.moe_gated_forward(s["x"], s["wg"], s["wu"], b["h"], b["workspace"], g=b["g"], u=b["u"])
    moe.moe_gated_backward(s["dh"], s["x"], s["wg"], s["wu"], b["g"], b["u"], b["dx"], b["dwg"], b["dwu"], b["workspace"])
    return {"h": b["h"], "dx": b["dx"], "dw_gate": b["dwg"], "dw_up": b["dwu"]}


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    b = _BYTES[case["type"]]
    held = lambda n: n * 17 / 32  # bytes of n values in MXFP4  # noqa: E731
    if case["op"] == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": 2 * b * n + held(n), "flops": 4 * n}
    if case["op"] == "product":
        r, n, k, e = case["rows"], case["N"], case["K"], case["E"]
        return {"bytes": held(r * k) + held(min(e, r) * n * k) + b * r * n, "flops": 2 * r * n * k}
    if case["op"] == "experts":
        t, h, f, e, top = case["T"], case["H"], case["F"], case["E"], case["top"]
        used = e * (1 - (1 - top / e) ** t)     # distinct experts of an even routing
        return {"bytes": 4 * t * h + held(3 * used * h * f) + b * t * top * h, "flops": 6 * t * top * h * f}
    t, h, f = case["T"], case["H"], case["F"]
    if not case["train"]:
        return {"bytes": b * (t * h + 2 * f * h + t * f), "flops": 4 * t * h * f}
    return {"bytes": b * (2 * t * h + 4 * f * h + 2 * t * f), "flops": 12 * t * h * f}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _power64(n):
    """2^n in 64 bits, exactly (whole n, in the normal range)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _quantised64(x):
    """The MXFP4 value of each entry of x (64 bits): the block's largest magnitude lies in
    [2^n, 2^(n+1)); in units of 2^(n-2) the entries are rounded half to even in steps of
    1/2 below 2, of 1 below 4 and of 2 up to 6."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().max(-1, keepdim=True).values
    n = (torch.where(top > 0, top, torch.ones_like(top)).view(torch.int64) >> 52) - 1023
    unit = _power64(n - 2)
    v = b / unit
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
    return ((torch.round(v / step) * step).clamp(-6, 6) * unit).flatten(-2)


def _held64(codes, scales):
    """Values of MXFP4 codes in 64 bits: sign bit, two exponent bits, one mantissa bit."""
    n = torch.stack([codes % 16, codes // 16], -1).flatten(-2).to(torch.int32)
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e > 0, (1 + m / 2) * _power64(e - 1), m / 2)
    mag = torch.where(n >= 8, -mag, mag).unflatten(-1, (-1, 32))
    return (mag * _power64(scales.long() - 127)[..., None]).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _quantised64(s["x"])
    if case["op"] in ("product", "experts"):
        ends = s["offsets"].tolist()
        out = []
        x = _held64(s["x"], s["xs"]) if case["op"] == "product" else _quantised64(s["x"])
        for e in range(case["E"]):
            if ends[e] == ends[e + 1]:
                continue
            if case["op"] == "product":
                out.append(x[ends[e]:ends[e + 1]] @ _held64(s["w"][e], s["ws"][e]).T)
                continue
            r = x[s["tok"][ends[e]:ends[e + 1]].long()]
            g, u, d = (_held64(s[k][0][e], s[k][1][e]) for k in ("wg", "wu", "wd"))
            p = r @ g.T
            out.append(_quantised64(p * torch.sigmoid(p) * (r @ u.T)) @ d.T)
        return torch.cat(out)
    x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
    g, u = x @ wg.T, x @ wu.T
    sig = torch.sigmoid(g)
    if not case["train"]:
        return g * sig * u
    dh = s["dh"].double()
    du = dh * g * sig
    dg = dh * u * (sig + g * sig * (1 - sig))
    return {"h": g * sig * u, "dx": dg @ wg + du @ wu, "dw_gate": dg.T @ x, "dw_up": du.T @ x}

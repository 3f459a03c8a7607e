"""Plain 64-bit forms of the operators around the expert layer, with bounds of what fp32 kernels may be off by.

Nothing here is shared with the library.  Bounds count roundings: a value held in a type is off by at most
eps/2 of it; a chain of n fp32 operations by at most n 2^-24 of the magnitudes that went in.  The kernels'
chains over a row are at most 16 additions in a thread, 5 between lanes and 16 between warps, and the formulas
add fewer than 40 operations: ROW and GRAD cover them.
"""
import torch

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}    # half of the smallest step, or more
U = 2.0 ** -24
ROW, GRAD = 96 * U, 256 * U


def inverse(v, eps):
    ms = v.square().mean(1, keepdim=True) + eps
    return torch.where(ms == 0, torch.zeros_like(ms), ms.clamp_min(1e-300).rsqrt())


def norm_forward(x, eps, y=None, post=None, gate=None, pre=None, a=1.0, b=1.0):
    """{name: (value, bound)} of 64-bit operands; gate as it broadcasts."""
    out, mag = a * x, abs(a) * x.abs()
    iy = torch.ones(x.shape[0], 1, dtype=x.dtype, device=x.device)
    if y is not None:
        z = y
        if post is not None:
            iy = inverse(y, eps)
            z = y * iy * post
        g = 1.0 if gate is None else gate
        out = out + b * g * z
        mag = mag + (b * g * z).abs()
    r = {"out": (out, ROW * mag), "iy": iy, "mag": mag, "io": torch.ones_like(iy)}
    if pre is not None:
        io = inverse(out, eps)
        n = out * io * pre
        rel = ROW * (1 + (mag * out.abs()).sum(1, keepdim=True) / out.square().sum(1, keepdim=True).clamp_min(1e-300))
        r["n"] = (n, (io * pre).abs() * ROW * mag + rel * n.abs())
        r["io"] = io
    return r


def norm_backward(x, eps, y=None, post=None, gate=None, pre=None, a=1.0, b=1.0, dout=None, dn=None):
    """{name: (gradient, bound)}; dgate in the gate's shape.  The bounds follow the kernel's sums, in which
    what cancels counts in full."""
    f = norm_forward(x, eps, y, post, gate, pre, a, b)
    out, mag, iy, io = f["out"][0], f["mag"], f["iy"], f["io"]
    H = x.shape[1]
    d = torch.zeros_like(x) if dout is None else dout.clone()
    dm = d.abs()
    r = {}
    if pre is not None:
        w = dn * pre
        d = d + io * w - out * io ** 3 * (w * out).sum(1, keepdim=True) / H
        dm = dm + (io * w).abs() + mag * io ** 3 * (w.abs() * mag).sum(1, keepdim=True) / H
        r["dpre"] = ((dn * out * io).sum(0), GRAD * (dn.abs() * mag * io).sum(0))
    r["dx"] = (a * d, GRAD * abs(a) * dm)
    if y is None:
        return r
    unit = y * iy
    z = unit if post is None else unit * post
    g = torch.ones(1, 1, dtype=x.dtype, device=x.device) if gate is None else gate
    if gate is not None:
        dg, dgm = b * d * z, abs(b) * dm * z.abs()
        for i in (0, 1):
            if g.shape[i] == 1 and x.shape[i] > 1:
                dg, dgm = dg.sum(i, keepdim=True), dgm.sum(i, keepdim=True)
        r["dgate"] = (dg, GRAD * dgm)
    dz, dzm = b * g * d, (b * g).abs() * dm
    if post is None:
        r["dy"] = (dz, GRAD * dzm)
        return r
    r["dpost"] = ((dz * unit).sum(0), GRAD * (dzm * unit.abs()).sum(0))
    c = (dz * post * y).sum(1, keepdim=True)
    cm = (dzm * (post * y).abs()).sum(1, keepdim=True)
    r["dy"] = (iy * (dz * post - iy ** 2 * c / H * y), GRAD * iy * (dzm * post.abs() + iy ** 2 * cm / H * y.abs()))
    return r


def balance(logits, ids, keff, offsets, K, valid=None, dloss=None, dw=None, norm=True, scale=1.0):
    """counts, tokens, loss and, with dloss or dw, the logits' gradient and its bound.  ids, keff, offsets, valid
    on the CPU as lists or tensors; one token at a time."""
    T, E = logits.shape
    l = logits.double()
    # log(sigmoid) normalised over the experts, so that scores far below zero keep their digits
    ls = torch.nn.functional.logsigmoid(l)
    top = ls.max(1, keepdim=True).values
    dead = top == -float("inf")
    p = torch.exp(ls - torch.where(dead, torch.zeros_like(top), top))
    p = torch.where(dead, torch.zeros_like(p), p / p.sum(1, keepdim=True).clamp_min(1e-300))
    rest, sig = torch.sigmoid(-l), torch.sigmoid(l)
    S = len(offsets) - 1
    counts, tokens = torch.zeros(S, E, dtype=torch.int64), torch.zeros(S, dtype=torch.int64)
    counted = torch.zeros(T, dtype=torch.bool)
    mean = torch.zeros(S, E, dtype=torch.float64)
    for s in range(S):
        for t in range(offsets[s], offsets[s + 1]):
            if valid is not None and not valid[t]:
                continue
            counted[t] = True
            tokens[s] += 1
            mean[s] += p[t]
            for i in range(min(max(int(keff[t]), 0), K)):
                if 0 <= int(ids[t][i]) < E:
                    counts[s, int(ids[t][i])] += 1
    n = max(int((tokens > 0).sum()), 1)
    f = counts.double() * E / counts.sum(1, keepdim=True).clamp_min(1)
    slope = f / (tokens.clamp_min(1)[:, None] * n)
    loss = (slope * mean).sum()
    # exp(-|l|) to 2 units and |l| roundings of its argument, quotient, the sums over E / 32 + 5 terms
    rel = (2 * l.abs().clamp_max(200).nan_to_num(posinf=200.0, neginf=200.0).amax(1, keepdim=True) + 64) * U
    loss_bound = float(loss.abs()) * (float(rel.max()) + (T / 8 + 700) * U)
    if dloss is None and dw is None:
        return counts, tokens, loss, loss_bound
    d, bound = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for s in range(S):
        for t in range(offsets[s], offsets[s + 1]):
            if not counted[t]:
                continue
            if dloss is not None:
                g = dloss * slope[s]
                dot = (g * p[t]).sum()
                d[t] += (g - dot) * p[t] * rest[t]
                bound[t] += (g.abs() + (g * p[t]).abs().sum()) * p[t] * rest[t] * 4 * rel[t]
            if dw is not None:
                kept = [i for i in range(min(max(int(keff[t]), 0), K)) if 0 <= int(ids[t][i]) < E]
                e = torch.tensor([int(ids[t][i]) for i in kept], dtype=torch.long)
                v = dw[t].double()[torch.tensor(kept, dtype=torch.long)]
                if not kept:
                    continue
                if norm:
                    best = ls[t, e].max()
                    h = torch.zeros_like(v) if best == -float("inf") else torch.softmax(ls[t, e], 0)
                    each = scale * h * rest[t, e] * (v - (h * v).sum())
                    mag = scale * h * rest[t, e] * (v.abs() + (h * v).abs().sum())
                else:
                    each = scale * sig[t, e] * rest[t, e] * v
                    mag = each.abs()
                d[t].index_add_(0, e, each)
                bound[t].index_add_(0, e, mag * 4 * rel[t])
    return counts, tokens, loss, loss_bound, d, bound


def adapter(x, down, up, scale, offsets, ids, y, base=None):
    """y (64 bits, changed in place) and the bound of the adapters' part: sums of K and R fp32 terms, whatever
    their order and whether additions round or truncate, and the R numbers between them held to 16 bits."""
    bound = torch.zeros_like(y)
    for s, a in enumerate(ids):
        p = slice(offsets[s], offsets[s + 1])
        had = 0.0 if base is None else base[p]
        y[p] = had
        if a >= 0:
            u, um = x[p] @ down[a].T, x[p].abs() @ down[a].abs().T
            c = 1.0 if scale is None else float(scale[a])
            y[p] = had + c * (u @ up[a].T)
            k, r = x.shape[1], up.shape[2]
            bound[p] = abs(c) * (((k * 2 * U + 2.0 ** -17) * um + 2 * (2 * r + 4) * U * u.abs()) @ up[a].abs().T)
            bound[p] += 4 * U * (y[p].abs() + abs(c) * (u.abs() @ up[a].abs().T))
    return y, bound

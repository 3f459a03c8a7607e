"""Train a dense gated block in 16 bits, convert it to MXFP4 and serve it, alone and as experts.

    python examples/dense_to_mxfp4.py [--tokens 256] [--hidden 512] [--d-ff 256] [--steps 60]

1. A dense block y = (silu(x Wg^T) * (x Wu^T)) Wd^T learns a teacher block of the same shape:
   moe_gated_forward and moe_gated_backward, the down projection by torch.
2. Its weights are converted with moe_quantize_mxfp4.
3. The converted block serves tokens: moe_mxfp4_expert_ffn without lists (a dense layer or a shared
   expert), and the same through moe_quantize_mxfp4 and moe_mxfp4_matmul for the down projection.
4. Copies of it, each with a few weights of its own, stand as the experts of a sparse layer:
   moe_route, moe_permute, moe_mxfp4_expert_ffn, moe_combine.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_expert_ffn_route_gb300 as moe  # noqa: E402


def rel(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def convert(w):
    """[.., n, k] -> MXFP4 codes [.., n, k/2] and scales [.., n, k/32]."""
    codes = torch.empty(*w.shape[:-1], w.shape[-1] // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(*w.shape[:-1], w.shape[-1] // 32, dtype=torch.uint8, device=w.device)
    moe.moe_quantize_mxfp4(w.contiguous(), codes, scales)
    return codes, scales


def block(x, wg, wu, wd):
    h = torch.empty(x.shape[0], wg.shape[0], dtype=x.dtype, device=x.device)
    moe.moe_gated_forward(x, wg, wu, h, moe.alloc_gated_workspace(x.shape[0], x.shape[1], wg.shape[0], False))
    return h, h @ wd.t()


def train(T, H, F, steps, g):
    """(weights in bf16, first loss, last loss) of a block that learns a random teacher."""
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5  # noqa: E731
    teacher = [rand(F, H).bfloat16(), rand(F, H).bfloat16(), rand(H, F).bfloat16()]
    master = [t.float() + 0.5 * rand(*t.shape) for t in teacher]
    state = [(torch.zeros_like(m), torch.zeros_like(m)) for m in master]
    ws = moe.alloc_gated_workspace(T, H, F, True)
    b16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h, gate, up, dx, dwg, dwu = b16(T, F), b16(T, F), b16(T, F), b16(T, H), b16(F, H), b16(F, H)
    losses = []
    for step in range(steps):
        x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        want = block(x, *teacher)[1].float()
        wg, wu, wd = (m.bfloat16() for m in master)
        moe.moe_gated_forward(x, wg, wu, h, ws, g=gate, u=up)
        err = (h @ wd.t()).float() - want
        losses.append(float(err.square().mean()))
        dy = (err * (2.0 / err.shape[0])).bfloat16()
        moe.moe_gated_backward(dy @ wd, x, wg, wu, gate, up, dx, dwg, dwu, ws)
        for m, (m1, m2), d in zip(master, state, (dwg, dwu, dy.t() @ h)):     # Adam
            d = d.float()
            m1.mul_(0.9).add_(d, alpha=0.1)
            m2.mul_(0.99).addcmul_(d, d, value=0.01)
            fix1, fix2 = 1 - 0.9 ** (step + 1), 1 - 0.99 ** (step + 1)
            m.addcdiv_(m1 / fix1, (m2 / fix2).sqrt() + 1e-8, value=-2e-3)
    moe.moe_check_errors(ws)
    return [m.bfloat16() for m in master], losses[0], losses[-1]


def serve_dense(weights, x):
    """The converted block in one call, and with its down projection apart."""
    wg, wu, wd = weights
    F, H = wg.shape
    T = x.shape[0]
    cfg = moe.MoeConfig.make(H, 1, 1, F)
    q = {}
    for k, w in (("gate", wg), ("up", wu), ("down", wd)):
        q["w_" + k], q["s_" + k] = convert(w[None])
    y = torch.empty(T, H, device="cuda")
    ws = moe.alloc_mxfp4_workspace(cfg, T)
    moe.moe_mxfp4_expert_ffn(cfg, x, q, y, ws)
    moe.moe_check_errors(ws)
    h = block(x, wg, wu, wd)[0]
    hq, hs = convert(h)
    y2, ws2 = torch.empty(T, H, device="cuda"), moe.alloc_mxfp4_matmul_workspace()
    moe.moe_mxfp4_matmul(hq, hs, q["w_down"][0], q["s_down"][0], y2, ws2)
    moe.moe_check_errors(ws2)
    return y, y2


def serve_experts(weights, x, E, K, g):
    """A sparse layer whose experts are E variants of the block: its output, and a plain one."""
    F, H = weights[0].shape
    T = x.shape[0]
    cfg = moe.MoeConfig.make(H, E, K, F)
    q, plain = {}, {}
    for k, w in zip(("gate", "up", "down"), weights):
        each = w.float()[None] * (1 + 0.05 * torch.randn(E, *w.shape, generator=g, device="cuda"))
        plain[k] = each
        q["w_" + k], q["s_" + k] = convert(each)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    xf, wr = x.float(), torch.randn(E, H, generator=g, device="cuda") / H ** 0.5
    ids, keff, wt = i32(T, K), i32(T), torch.empty(T, K, device="cuda")
    counts, off, tok, slot, uniq, nu = i32(E), i32(E + 1), i32(T * K), i32(T * K), i32(E), i32(1)
    ws, ms = moe.alloc_workspace(cfg, T), moe.alloc_mxfp4_workspace(cfg, T)
    pairs, y = torch.empty(T * K, H, device="cuda"), torch.empty(T, H, device="cuda")
    moe.moe_route(cfg, xf, wr, torch.zeros(E, device="cuda"), ids, wt, keff, ws)
    moe.moe_permute(cfg, ids, keff, counts, off, tok, slot, uniq, nu, ws)
    moe.moe_mxfp4_expert_ffn(cfg, xf, q, pairs, ms, offsets=off, tok=tok)
    moe.moe_combine(cfg, pairs, ids, keff, wt, off, tok, y, ws)
    moe.moe_check_errors(ws)
    moe.moe_check_errors(ms)
    want = torch.zeros_like(y)
    for e in range(E):
        h = torch.nn.functional.silu(xf @ plain["gate"][e].t()) * (xf @ plain["up"][e].t())
        want += (wt * (ids == e)).sum(1, keepdim=True) * (h @ plain["down"][e].t())
    return y, want


def main(tokens=256, hidden=512, d_ff=256, steps=60, experts=8, top_k=2, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    weights, first, last = train(tokens, hidden, d_ff, steps, g)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    y16 = block(x, *weights)[1]
    y, y2 = serve_dense(weights, x)
    ys, want = serve_experts(weights, x, experts, top_k, g)
    out = {"first_loss": first, "last_loss": last, "mxfp4_block": rel(y, y16), "mxfp4_down": rel(y2, y16),
           "mxfp4_experts": rel(ys, want)}
    print("loss %.4f -> %.4f over %d steps; relative error in MXFP4: block %.3f, down projection alone %.3f, "
          "sparse layer of %d experts %.3f" % (first, last, steps, out["mxfp4_block"], out["mxfp4_down"], experts,
                                               out["mxfp4_experts"]))
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 256), ("hidden", 512), ("d-ff", 256), ("steps", 60)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    main(a.tokens, a.hidden, a.d_ff, a.steps)

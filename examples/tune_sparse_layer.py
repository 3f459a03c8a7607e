"""Tune what stands around a sparse layer with frozen MXFP4 experts, then serve it with adapters.

    python examples/tune_sparse_layer.py [--tokens 256] [--hidden 256] [--d-ff 128] [--experts 16] [--steps 20]

1. A step: the norm ahead of the block (moe_block_norm_forward), the router (moe_route) and how evenly it loads the
   experts (moe_balance_forward), the experts (moe_permute, moe_mxfp4_expert_ffn, moe_combine), and the block's way
   back into the residual stream with its own norm and a learned scale a channel.
2. Its gradients: moe_block_norm_backward, the applied weights' from the experts' outputs, and from those and the
   balance loss the router's logits' (moe_balance_backward).  The experts are frozen; what they pass on to their
   input is left out.
3. Served: a projection that all requests share (moe_mxfp4_matmul) and beside it each request's own adapter
   (moe_adapter_matmul), added in place.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_expert_ffn_route_gb300 as moe  # noqa: E402

EPS = 1e-5


def convert(w):
    """[.., n, k] -> MXFP4 codes [.., n, k/2] and scales [.., n, k/32]."""
    codes = torch.empty(*w.shape[:-1], w.shape[-1] // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(*w.shape[:-1], w.shape[-1] // 32, dtype=torch.uint8, device=w.device)
    moe.moe_quantize_mxfp4(w.contiguous(), codes, scales)
    return codes, scales


class Layer:
    """A sparse layer between two norms: its parameters, frozen experts and buffers for T tokens."""

    def __init__(self, T, H, F, E, K, g):
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.cfg = moe.MoeConfig.make(H, E, K, F, routed_scaling_factor=2.0)
        self.p = {"pre": 1 + 0.1 * rand(H), "post": 1 + 0.1 * rand(H), "gate": 0.5 + 0.1 * rand(H), "router": rand(E, H) / H ** 0.5}
        self.bias = torch.zeros(E, device="cuda")
        self.experts = {}
        for name, shape in (("gate", (E, F, H)), ("up", (E, F, H)), ("down", (E, H, F))):
            self.experts["w_" + name], self.experts["s_" + name] = convert(rand(*shape) / shape[-1] ** 0.5)
        self.ids, self.keff, self.w = i32(T, K), i32(T), f32(T, K)
        self.lists = (i32(E), i32(E + 1), i32(T * K), i32(T * K), i32(E), i32(1))     # counts .. n_uniq
        self.n, self.pairs, self.y, self.out = f32(T, H), f32(T * K, H), f32(T, H), f32(T, H)
        self.kept, self.kept_in = f32(T, 2), f32(T, 2)
        self.ws, self.mx = moe.alloc_workspace(self.cfg, T), moe.alloc_mxfp4_workspace(self.cfg, T)
        self.norm_ws = moe.alloc_block_norm_workspace(T, H)

    def forward(self, x, offsets):
        """(out, balance loss) of tokens x [T][H] in sequences."""
        p, cfg, S = self.p, self.cfg, offsets.numel() - 1
        moe.moe_block_norm_forward(x, EPS, pre_w=p["pre"], n=self.n, kept=self.kept_in)
        moe.moe_route(cfg, self.n, p["router"], self.bias, self.ids, self.w, self.keff, self.ws)
        self.logits = self.n @ p["router"].t()
        self.loss, self.counts = torch.empty(1, device="cuda"), torch.empty(S, cfg.n_experts, dtype=torch.int32, device="cuda")
        self.tokens = torch.empty(S, dtype=torch.int32, device="cuda")
        self.bal_ws = moe.alloc_balance_workspace(cfg, x.shape[0], S)
        moe.moe_balance_forward(cfg, self.logits, self.ids, self.keff, offsets, self.loss, self.counts, self.tokens, self.bal_ws)
        _, off, tok, _, _, _ = self.lists
        moe.moe_permute(cfg, self.ids, self.keff, *self.lists, self.ws)
        moe.moe_mxfp4_expert_ffn(cfg, self.n, self.experts, self.pairs, self.mx, offsets=off, tok=tok)
        moe.moe_combine(cfg, self.pairs, self.ids, self.keff, self.w, off, tok, self.y, self.ws)
        moe.moe_block_norm_forward(x, EPS, y=self.y, post_w=p["post"], gate=p["gate"], out=self.out, kept=self.kept)
        return self.out, self.loss

    def backward(self, x, offsets, dout, dloss):
        """Gradients of the parameters and of x."""
        p, T, H = self.p, *x.shape
        g = {k: torch.empty_like(p[k]) for k in ("pre", "post", "gate")}
        dx, dy, back = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        moe.moe_block_norm_backward(x, self.kept, self.norm_ws, y=self.y, post_w=p["post"], gate=p["gate"], dout=dout, dx=dx, dy=dy,
                                    dgate=g["gate"], dpost=g["post"])
        # the gradient of an applied weight: its expert's output times the combined output's gradient
        slot = self.lists[3].long()
        dw = torch.zeros(T * self.cfg.top_k, device="cuda")
        dw[slot] = (self.pairs * dy[slot // self.cfg.top_k]).sum(1)
        dl = torch.empty_like(self.logits)
        moe.moe_balance_backward(self.cfg, self.logits, self.ids, self.keff, offsets, self.counts, self.tokens, dl, self.bal_ws,
                                 dloss=dloss, dw=dw.view(T, -1))
        g["router"] = dl.t() @ self.n
        moe.moe_block_norm_backward(x, self.kept_in, self.norm_ws, pre_w=p["pre"], dn=dl @ p["router"], dx=back, dpre=g["pre"])
        for ws in (self.ws, self.mx, self.norm_ws, self.bal_ws):
            moe.moe_check_errors(ws)
        return g, dx + back


def serve(h, weight, down, up, scale, offsets, ids):
    """y = h weight^T, and in place each segment's adapter; h bfloat16, weight in MXFP4."""
    N = weight[0].shape[0]
    y = torch.empty(h.shape[0], N, device="cuda")
    codes, scales = convert(h)
    ws, aw = moe.alloc_mxfp4_matmul_workspace(), moe.alloc_adapter_workspace(h.shape[0], down.shape[1])
    moe.moe_mxfp4_matmul(codes, scales, *weight, y, ws)
    shared = y.clone()
    moe.moe_adapter_matmul(h, down, up, scale, offsets, ids, y, aw, base=y)
    moe.moe_check_errors(ws)
    moe.moe_check_errors(aw)
    return shared, y


def main(tokens=256, hidden=256, d_ff=128, experts=16, top_k=4, steps=20, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    layer = Layer(tokens, hidden, d_ff, experts, top_k, g)
    teacher = Layer(tokens, hidden, d_ff, experts, top_k, g)
    teacher.experts = layer.experts
    offsets = torch.tensor([0, tokens // 3, tokens], dtype=torch.int32, device="cuda")
    dloss = torch.full((1,), 0.01, device="cuda")
    history = []
    for _ in range(steps):
        x = rand(tokens, hidden)
        want = teacher.forward(x, offsets)[0]
        out, balance = layer.forward(x, offsets)
        err = out - want
        history.append((float(err.square().mean()), float(balance)))
        grads, _ = layer.backward(x, offsets, err * (2.0 / err.numel()), dloss)
        for k, v in layer.p.items():
            v -= 1e-3 * grads[k].sign()
    for i in (0, -1):
        print("step %d: squared error %.4f, balance loss %.3f" % (i % steps, *history[i]))
    h = rand(tokens, d_ff).bfloat16()
    weight = convert(rand(hidden, d_ff) / d_ff ** 0.5)
    down, up = (rand(3, 16, d_ff) / d_ff ** 0.5).bfloat16(), (rand(3, hidden, 16) / 4).bfloat16()
    ends = torch.tensor([0, 1, 2, tokens // 2, tokens], dtype=torch.int32, device="cuda")
    ids = torch.tensor([2, 0, -1, 1], dtype=torch.int32, device="cuda")
    shared, y = serve(h, weight, down, up, torch.ones(3, device="cuda"), ends, ids)
    print("adapters: mean change %.3f of the shared projection's %.3f" % (float((y - shared).abs().mean()), float(shared.abs().mean())))
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 256), ("hidden", 256), ("d-ff", 128), ("experts", 16), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    main(a.tokens, a.hidden, a.d_ff, a.experts, steps=a.steps)

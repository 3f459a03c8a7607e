"""The operators around a sparse layer together, as the example uses them: its gradients against automatic ones in
64 bits, and its serving against the plain form."""
import os
import sys

import pytest
import torch

import plain_around as pa
import sparse_expert_ffn_route_gb300 as moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def rms(v, w):
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-5) * w


def test_a_step():
    import tune_sparse_layer as ex
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, E, K = 70, 128, 12, 3
    layer = ex.Layer(T, H, 64, E, K, g)
    x = torch.randn(T, H, generator=g, device="cuda")
    off = [0, 9, 9, T]
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    out, loss = layer.forward(x, offsets)
    dout, dloss = torch.randn(T, H, generator=g, device="cuda"), torch.tensor([0.3], device="cuda")
    grads, dx = layer.backward(x, offsets, dout, dloss)

    # the same step in 64 bits, with the library's choice of experts and its experts' outputs as constants
    p = {k: v.double().requires_grad_() for k, v in layer.p.items()}
    xd = x.double().requires_grad_()
    n = rms(xd, p["pre"])
    sig = torch.sigmoid(n @ p["router"].t())
    kept = torch.gather(sig, 1, layer.ids.long())
    w = 2.0 * kept / kept.sum(1, keepdim=True)
    pairs = torch.empty(T * K, H, dtype=torch.float64, device="cuda")
    pairs[layer.lists[3].long()] = layer.pairs.double()           # by token and place
    y = (w[:, :, None] * pairs.view(T, K, H)).sum(1)
    want = xd + p["gate"] * rms(y, p["post"])
    share = sig / sig.sum(1, keepdim=True)
    balance = 0.0
    for a, b in zip(off, off[1:]):
        if a < b:
            load = torch.bincount(layer.ids[a:b].flatten().long(), minlength=E).double()
            balance = balance + (load * E / load.sum() * share[a:b].mean(0)).sum() / 2
    ((want * dout).sum() + 0.3 * balance).backward()

    # fp32 chains of about H + T + 300 operations, each off by 2^-24 of what goes in; what cancels grows by less
    # than ten times (norms, weights and shares are differences of terms of their own size)
    limit = 10 * (H + T + 300) * pa.U

    def close(got, exact, what):
        assert float((got.double() - exact).norm() / exact.norm()) <= limit, what
    close(out, want.detach(), "out")
    close(loss, balance.detach().reshape(1), "loss")
    for k, v in grads.items():
        close(v, p[k].grad, k)
    close(dx, xd.grad, "x")


@pytest.mark.parametrize("T,ends,ids", [(6, [0, 1, 2, 3, 6], [2, 0, -1, 2]), (300, [0, 1, 140, 150, 300], [1, 0, -1, 2])])
def test_serving(T, ends, ids):
    import tune_sparse_layer as ex
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, weight = rand(T, 512).bfloat16(), ex.convert(rand(264, 512) / 512 ** 0.5)
    down, up, scale = (rand(3, 16, 512) / 512 ** 0.5).bfloat16(), (rand(3, 264, 16) / 4).bfloat16(), rand(3)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    shared, y = ex.serve(h, weight, down, up, scale, i32(ends), i32(ids))
    want, bound = pa.adapter(h.double(), down.double(), up.double(), scale, ends, ids, torch.zeros_like(y, dtype=torch.float64),
                             shared.double())
    assert bool(((y.double() - want).abs() <= bound + 2 * pa.U * (want.abs() + bound)).all())


def test_the_example_runs():
    import tune_sparse_layer as ex
    history = ex.main(tokens=96, hidden=128, d_ff=64, experts=8, top_k=2, steps=3)
    assert len(history) == 3 and all(e == e and b >= 0.5 for e, b in history)


def test_two_streams_at_once():
    """The same calls on two streams, each with its own workspaces."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, K, N = 700, 512, 520
    x, down, up = rand(T, K).bfloat16(), rand(2, 16, K).bfloat16(), rand(2, N, 16).bfloat16()
    off, ids = torch.tensor([0, 300, T], dtype=torch.int32, device="cuda"), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    stream, y, post = rand(T, N), rand(T, N).bfloat16(), 1 + rand(N)

    def call(to, ws, nws):
        moe.moe_adapter_matmul(x, down, up, None, off, ids, to["y"], ws)
        moe.moe_block_norm_forward(stream, 1e-5, y=y, post_w=post, pre_w=post, out=to["out"], n=to["n"], kept=to["kept"])
        moe.moe_block_norm_backward(stream, to["kept"], nws, y=y, post_w=post, pre_w=post, dout=stream, dn=y, dx=to["dx"], dy=to["dy"],
                                    dpost=to["dpost"], dpre=to["dpre"])

    def buffers():
        e = torch.empty
        return {"y": e(T, N, device="cuda"), "out": e(T, N, device="cuda"), "n": e(T, N, device="cuda", dtype=torch.bfloat16),
                "kept": e(T, 2, device="cuda"), "dx": e(T, N, device="cuda"), "dy": e(T, N, device="cuda", dtype=torch.bfloat16),
                "dpost": e(N, device="cuda"), "dpre": e(N, device="cuda")}
    want, ws, nws = buffers(), moe.alloc_adapter_workspace(T, 16), moe.alloc_block_norm_workspace(T, N)
    call(want, ws, nws)
    torch.cuda.synchronize()
    sides = [(torch.cuda.Stream(), buffers(), moe.alloc_adapter_workspace(T, 16), moe.alloc_block_norm_workspace(T, N)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, to, a, b in sides:
            with torch.cuda.stream(s):
                call(to, a, b)
    torch.cuda.synchronize()
    for _, to, a, b in sides:
        moe.moe_check_errors(a)
        moe.moe_check_errors(b)
        for k, v in want.items():
            assert torch.equal(v, to[k]), k

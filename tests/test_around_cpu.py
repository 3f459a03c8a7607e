"""What the calls around the expert layer refuse, on the host: in the binding, and in the library before anything is
enqueued.  And the plain gradients against automatic ones and differences."""
import ctypes

import pytest
import torch

import plain_around as pa
import sparse_expert_ffn_route_gb300 as moe
from sparse_expert_ffn_route_gb300 import binding
from test_mxfp4_binding_cpu import Called, NoStream, OnDevice, bound  # noqa: F401

FAKE = 1 << 20
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
CFG = moe.MoeConfig.make(64, 16, 2, 64)


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def calls():
    """name -> (function of keyword tensors, its tensors)"""
    s = NoStream
    ws = OnDevice(1 << 20, dtype=U8)
    return {
        "norm": (lambda **t: moe.moe_block_norm_forward(eps=1e-5, **t, stream=s),
                 dict(x=OnDevice(4, 64, dtype=F32), y=OnDevice(4, 64), post_w=OnDevice(64, dtype=F32), gate=OnDevice(4, 64),
                      pre_w=OnDevice(64, dtype=F32), out=OnDevice(4, 64, dtype=F32), n=OnDevice(4, 64), kept=OnDevice(4, 2, dtype=F32))),
        "norm_back": (lambda **t: moe.moe_block_norm_backward(**t, stream=s),
                      dict(x=OnDevice(4, 64, dtype=F32), kept=OnDevice(4, 2, dtype=F32), workspace=ws, y=OnDevice(4, 64),
                           post_w=OnDevice(64, dtype=F32), gate=OnDevice(4, 1), pre_w=OnDevice(64, dtype=F32),
                           dout=OnDevice(4, 64, dtype=F32), dn=OnDevice(4, 64), dx=OnDevice(4, 64, dtype=F32), dy=OnDevice(4, 64),
                           dgate=OnDevice(4, 1, dtype=F32), dpost=OnDevice(64, dtype=F32), dpre=OnDevice(64, dtype=F32))),
        "balance": (lambda **t: moe.moe_balance_forward(CFG, **t, stream=s),
                    dict(logits=OnDevice(4, 16), ids=OnDevice(4, 2, dtype=I32), keff=OnDevice(4, dtype=I32),
                         seq_offsets=OnDevice(3, dtype=I32), loss=OnDevice(1, dtype=F32), counts=OnDevice(2, 16, dtype=I32),
                         tokens=OnDevice(2, dtype=I32), workspace=ws, valid=OnDevice(4, dtype=U8))),
        "balance_back": (lambda **t: moe.moe_balance_backward(CFG, **t, stream=s),
                         dict(logits=OnDevice(4, 16), ids=OnDevice(4, 2, dtype=I32), keff=OnDevice(4, dtype=I32),
                              seq_offsets=OnDevice(3, dtype=I32), counts=OnDevice(2, 16, dtype=I32), tokens=OnDevice(2, dtype=I32),
                              dlogits=OnDevice(4, 16), workspace=ws, dloss=OnDevice(1, dtype=F32), dw=OnDevice(4, 2, dtype=F32),
                              valid=OnDevice(4, dtype=U8))),
        "adapter": (lambda **t: moe.moe_adapter_matmul(**t, stream=s),
                    dict(x=OnDevice(4, 64), down=OnDevice(3, 8, 64), up=OnDevice(3, 32, 8), scale=OnDevice(3, dtype=F32),
                         offsets=OnDevice(3, dtype=I32), ids=OnDevice(2, dtype=I32), y=OnDevice(4, 32, dtype=F32), workspace=ws,
                         base=OnDevice(4, 32, dtype=F32))),
    }


NAMES = ("norm", "norm_back", "balance", "balance_back", "adapter")


@pytest.mark.parametrize("name", NAMES)
def test_right_tensors_reach_the_library(bound, name):  # noqa: F811
    call, tensors = calls()[name]
    with pytest.raises(Called):
        call(**tensors)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("bad", [dict(device=-1), dict(device=1), dict(dtype=torch.float64), "contiguous", "shape"])
def test_every_tensor_is_checked(bound, name, bad):  # noqa: F811
    """On the same device, of its type, dense (x and y may have strided rows) and of its shape."""
    call, tensors = calls()[name]
    for k, t in tensors.items():
        if bad == "contiguous":
            if k in ("x", "logits") or (k == "y" and name.startswith("norm")):
                continue
            other = OnDevice(*t.shape, dtype=t.dtype, contiguous=False)
        elif bad == "shape":
            if k == "workspace" or (k == "ids" and name == "adapter"):   # any size; the segments' number
                continue
            other = OnDevice(*t.shape[:-1], t.shape[-1] + 8, dtype=t.dtype)
        else:
            other = OnDevice(*t.shape, **{"dtype": t.dtype, **bad})
        with pytest.raises(ValueError):
            call(**{**tensors, k: other})


@pytest.mark.parametrize("name", NAMES)
def test_the_device_is_the_current_one(bound, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    call, tensors = calls()[name]
    with pytest.raises(ValueError, match="current device"):
        call(**tensors)


def test_gates_by_shape(bound):  # noqa: F811
    gate = lambda g, T, d=None: binding._gate(g, d, T, 64, BF16, 0)[1]  # noqa: E731
    assert gate(None, 4) == moe.MOE_GATE_NONE
    assert gate(OnDevice(64), 4) == gate(OnDevice(1, 64), 4) == moe.MOE_GATE_CHANNEL
    assert gate(OnDevice(4, 1), 4) == gate(OnDevice(1, 1), 1) == moe.MOE_GATE_TOKEN
    assert gate(OnDevice(4, 64), 4) == gate(OnDevice(1, 64), 1) == gate(OnDevice(1, 64), 1, OnDevice(1, 64)) == moe.MOE_GATE_FULL
    assert gate(OnDevice(1, 64), 1, OnDevice(1, 64, dtype=F32)) == moe.MOE_GATE_CHANNEL
    for bad in (OnDevice(4), OnDevice(64, 1), OnDevice(4, 32), OnDevice(2, 64)):
        with pytest.raises(ValueError, match="gate"):
            gate(bad, 4)
    call, tensors = calls()["norm_back"]
    with pytest.raises(ValueError, match="gate"):
        call(**{**tensors, "gate": None})


def ready(rc):
    """The arguments are right: without a GPU the library then says that there is none."""
    return torch.cuda.is_available() or rc == moe.MOE_ERR_UNSUPPORTED


def test_norm_refusals(lib):
    names = ("x", "ldx", "xd", "y", "ldy", "gate", "kind", "dt", "post", "pre", "eps", "a", "b", "T", "H", "out", "n", "kept", "st")
    ok = [FAKE, 64, 0, FAKE, 64, FAKE, 1, 1, FAKE, FAKE, 1e-5, 1.0, 1.0, 4, 64, FAKE, FAKE, FAKE, None]

    def fwd(**kw):
        return lib.moe_block_norm_forward(*[kw.get(k, v) for k, v in zip(names, ok)])
    A, S, L = moe.MOE_ERR_ARG, moe.MOE_ERR_SHAPE, moe.MOE_ERR_ALIGN
    if not torch.cuda.is_available():
        assert ready(fwd()) and ready(fwd(gate=None, kind=0)) and ready(fwd(out=None)) and ready(fwd(pre=None, n=None))
        assert ready(fwd(y=None, gate=None, kind=0, post=None)) and ready(fwd(kept=None)) and ready(fwd(gate=FAKE + 2, kind=2))
    assert fwd(x=None) == A and fwd(y=None) == A and fwd(gate=None) == A and fwd(kind=0) == A and fwd(kind=4) == A
    assert fwd(n=None) == A and fwd(pre=None) == A and fwd(pre=None, n=None, out=None) == A
    assert fwd(xd=3) == A and fwd(dt=-1) == A
    for bad in (-1.0, float("inf"), float("nan")):
        assert fwd(eps=bad) == A
    assert fwd(a=float("nan")) == A and fwd(b=float("inf")) == A
    assert fwd(T=-1) == S and fwd(T=(1 << 24) + 1) == S and fwd(T=0, x=None) == moe.MOE_OK
    assert fwd(H=60) == S and fwd(H=0) == S and fwd(H=8200) == S
    assert fwd(ldx=56) == S and fwd(ldy=0) == S and fwd(ldx=66) == L and fwd(ldy=68) == L
    for k in ("x", "y", "gate", "post", "pre", "out", "n", "kept"):
        assert fwd(**{k: FAKE + 4}) == L, k
    need = moe.moe_block_norm_workspace_size(4, 64)
    assert need > 256 and not moe.moe_block_norm_workspace_size(4, 60) and not moe.moe_block_norm_workspace_size(-1, 64)
    sizes = [moe.moe_block_norm_workspace_size(t, 1024) for t in (0, 1, 10, 100, 100000)]
    assert sizes == sorted(sizes)
    names = ("x", "ldx", "xd", "y", "ldy", "gate", "kind", "dt", "post", "pre", "kept", "a", "b", "T", "H", "dout", "dn", "dx", "dy",
             "dgate", "dpost", "dpre", "ws", "bytes", "st")
    ok2 = [FAKE, 64, 0, FAKE, 64, FAKE, 3, 1, FAKE, FAKE, FAKE, 1.0, 1.0, 4, 64] + [FAKE] * 8 + [need, None]

    def bwd(**kw):
        return lib.moe_block_norm_backward(*[kw.get(k, v) for k, v in zip(names, ok2)])
    if not torch.cuda.is_available():
        assert ready(bwd()) and ready(bwd(dout=None)) and ready(bwd(dn=None, pre=None, dpre=None))
        assert ready(bwd(**dict.fromkeys(("dx", "dy", "dgate", "dpost", "dpre"))))
    assert bwd(x=None) == A and bwd(kept=None) == A and bwd(dn=None) == A and bwd(pre=None) == A
    assert bwd(dout=None, dn=None, pre=None, dpre=None) == A and bwd(y=None, gate=None, kind=0, post=None) == A
    assert bwd(post=None) == A and bwd(gate=None, kind=0) == A
    for k in ("dout", "dn", "dx", "dy", "dgate", "dpost", "dpre", "kept"):
        assert bwd(**{k: FAKE + 4}) == L, k
    assert bwd(ws=None) == moe.MOE_ERR_WORKSPACE and bwd(ws=FAKE + 128) == L and bwd(bytes=need - 1) == moe.MOE_ERR_WORKSPACE
    assert bwd(T=0, dgate=None, dpost=None, dpre=None, ws=None) == moe.MOE_OK


def test_balance_refusals(lib):
    names = ("cfg", "logits", "dt", "ld", "ids", "keff", "T", "off", "S", "valid", "loss", "counts", "tokens", "ws", "bytes", "st")
    need = moe.moe_balance_workspace_size(CFG, 4, 2)
    ok = [ctypes.byref(CFG), FAKE, 1, 16, FAKE, FAKE, 4, FAKE, 2, FAKE, FAKE, FAKE, FAKE, FAKE, need, None]

    def fwd(**kw):
        return lib.moe_balance_forward(*[kw.get(k, v) for k, v in zip(names, ok)])
    A, S, L, W = moe.MOE_ERR_ARG, moe.MOE_ERR_SHAPE, moe.MOE_ERR_ALIGN, moe.MOE_ERR_WORKSPACE
    if not torch.cuda.is_available():
        assert ready(fwd()) and ready(fwd(valid=None)) and ready(fwd(valid=FAKE + 1)) and ready(fwd(logits=FAKE + 2))
        assert ready(fwd(T=0, logits=None, ids=None, keff=None))
    for k in ("cfg", "logits", "ids", "keff", "off", "loss", "counts", "tokens"):
        assert fwd(**{k: None}) == A, k
    for k in ("logits", "ids", "keff", "off", "loss", "counts", "tokens"):
        assert fwd(**{k: FAKE + 1}) == L, k
    assert fwd(dt=5) == A and fwd(ld=15) == S and fwd(T=-1) == S and fwd(S=0) == S and fwd(S=(1 << 20) + 1) == S
    assert fwd(cfg=ctypes.byref(moe.MoeConfig.make(64, 600, 2, 64))) == S
    assert fwd(ws=None) == W and fwd(bytes=need - 1) == W and fwd(ws=FAKE + 16) == L
    size = moe.moe_balance_workspace_size
    assert not size(CFG, -1, 1) and not size(CFG, 4, 0)
    for cfg, most in ((CFG, 20000), (moe.MoeConfig.make(64, 384, 8, 64), 70000)):   # one for more tokens serves fewer
        sizes = [size(cfg, t, 3) for t in range(0, most, 997)]
        assert sizes == sorted(sizes)
    names = ("cfg", "logits", "dt", "ld", "ids", "keff", "T", "off", "S", "valid", "counts", "tokens", "dloss", "dw", "d", "gdt", "ws",
             "bytes", "st")
    ok2 = [ctypes.byref(CFG), FAKE, 1, 16, FAKE, FAKE, 4, FAKE, 2, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, FAKE, 256, None]

    def bwd(**kw):
        return lib.moe_balance_backward(*[kw.get(k, v) for k, v in zip(names, ok2)])
    if not torch.cuda.is_available():
        assert ready(bwd()) and ready(bwd(dw=None)) and ready(bwd(dloss=None)) and ready(bwd(gdt=0))
    assert bwd(dloss=None, dw=None) == A and bwd(d=None) == A and bwd(gdt=2) == A and bwd(dt=0, gdt=1) == A
    assert bwd(dloss=FAKE + 2) == L and bwd(d=FAKE + 1) == L and bwd(bytes=255) == W and bwd(T=0) == moe.MOE_OK


def test_adapter_refusals(lib):
    names = ("x", "ldx", "dt", "T", "K", "down", "up", "scale", "A", "R", "N", "off", "ids", "S", "base", "y", "yd", "ws", "bytes", "st")
    need = moe.moe_adapter_workspace_size(4, 8)
    ok = [FAKE, 64, 1, 4, 64, FAKE, FAKE, FAKE, 3, 8, 32, FAKE, FAKE, 2, FAKE, FAKE, 0, FAKE, need, None]

    def call(**kw):
        return lib.moe_adapter_matmul(*[kw.get(k, v) for k, v in zip(names, ok)])
    A, S, L, W = moe.MOE_ERR_ARG, moe.MOE_ERR_SHAPE, moe.MOE_ERR_ALIGN, moe.MOE_ERR_WORKSPACE
    if not torch.cuda.is_available():
        assert ready(call()) and ready(call(base=None)) and ready(call(scale=None)) and ready(call(T=1 << 20))
    for k in ("x", "down", "up", "off", "ids", "y"):
        assert call(**{k: None}) == A, k
    for k in ("x", "down", "up", "off", "ids", "y", "base", "scale"):
        assert call(**{k: FAKE + 2}) == L, k
    assert call(dt=0) == A and call(yd=4) == A
    assert call(T=-1) == S and call(T=0) == moe.MOE_OK and call(K=60) == S and call(N=4) == S and call(ldx=56) == S and call(ldx=68) == L
    for r in (0, 4, 12, 136):
        assert call(R=r) == S
    assert call(A=0) == S and call(A=(1 << 16) + 1) == S and call(S=0) == S and call(A=1 << 16, N=1 << 16) == S
    assert call(ws=None) == W and call(bytes=need - 1) == W and call(ws=FAKE + 64) == L
    size = moe.moe_adapter_workspace_size
    assert size(0, 8) == 256 and not size(4, 7) and not size(-1, 8) and size(4, 8) == size(128, 8) < size(129, 8)


@pytest.mark.parametrize("gate", [None, (1, 24), (6, 1), (6, 24)])
def test_plain_norm_gradients(gate):
    g = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    leaves = {"x": rand(6, 24), "y": rand(6, 24), "post": rand(24), "pre": rand(24)} | ({} if gate is None else {"gate": rand(*gate)})
    for t in leaves.values():
        t.requires_grad_()
    dout, dn = rand(6, 24), rand(6, 24)

    def value(v):
        f = pa.norm_forward(v["x"], 1e-3, v["y"], v["post"], v.get("gate"), v["pre"], 0.7, 1.3)
        return (f["out"][0] * dout).sum() + (f["n"][0] * dn).sum()
    value(leaves).backward()
    plain = {k: t.detach() for k, t in leaves.items()}
    r = pa.norm_backward(plain["x"], 1e-3, plain["y"], plain["post"], plain.get("gate"), plain["pre"], 0.7, 1.3, dout, dn)
    for k, t in leaves.items():
        got = r["d" + k][0]
        assert torch.allclose(got, t.grad, rtol=1e-11, atol=1e-12), k
        step = rand(*t.shape)      # and along a direction, by differences
        h = 1e-6
        up, down = dict(plain), dict(plain)
        up[k], down[k] = plain[k] + h * step, plain[k] - h * step
        assert abs(float((value(up) - value(down)) / (2 * h) - (got * step).sum())) < 1e-6


@pytest.mark.parametrize("norm", [True, False])
def test_plain_balance_gradient(norm):
    g = torch.Generator().manual_seed(2)
    T, E, K, off = 9, 7, 3, [0, 4, 4, 9]
    l = torch.randn(T, E, generator=g, dtype=torch.float64)
    ids = torch.rand(T, E, generator=g).topk(K, dim=1)[1]
    keff = torch.randint(0, K + 1, (T,), generator=g)
    valid = torch.tensor([1, 1, 0, 1, 1, 1, 1, 0, 1])
    dw = torch.randn(T, K, generator=g, dtype=torch.float64)
    counts, tokens, loss, _, d, _ = pa.balance(l, ids, keff, off, K, valid, 0.7, dw, norm, 2.5)
    assert tokens.tolist() == [3, 0, 4]
    x = l.clone().requires_grad_()
    sig = torch.sigmoid(x)
    p = sig / sig.sum(1, keepdim=True)
    total = torch.zeros((), dtype=torch.float64)
    for s in (0, 2):
        rows = [t for t in range(off[s], off[s + 1]) if valid[t]]
        f = E * counts[s].double() / counts[s].sum()
        total = total + (f * p[rows].mean(0)).sum() / 2
    assert abs(float(total.detach()) - float(loss)) < 1e-12
    weights = torch.zeros((), dtype=torch.float64)
    for t in range(T):
        k = int(keff[t]) if valid[t] else 0
        if k:
            w = sig[t, ids[t, :k]]
            weights = weights + (2.5 * (w / w.sum() if norm else w) * dw[t, :k]).sum()
    (0.7 * total + weights).backward()
    assert torch.allclose(d, x.grad, rtol=1e-10, atol=1e-13)


def test_norm_in_place_needs_dense_rows(lib):
    """out and n are dense: x or y with rows further apart cannot hold them."""
    names = ("x", "ldx", "xd", "y", "ldy", "gate", "kind", "dt", "post", "pre", "eps", "a", "b", "T", "H", "out", "n", "kept", "st")
    X, Y, O, N = (FAKE * i for i in (1, 2, 3, 4))
    ok = [X, 64, 0, Y, 64, None, 0, 1, None, FAKE * 5, 1e-5, 1.0, 1.0, 4, 64, O, N, None, None]

    def fwd(**kw):
        return lib.moe_block_norm_forward(*[kw.get(k, v) for k, v in zip(names, ok)])
    if not torch.cuda.is_available():
        assert ready(fwd()) and ready(fwd(out=X, n=Y)) and ready(fwd(ldx=72, ldy=72))
        assert ready(fwd(out=X, n=Y, T=1, ldx=72, ldy=72))
    assert fwd(out=X, ldx=72) == moe.MOE_ERR_ARG and fwd(n=Y, ldy=72) == moe.MOE_ERR_ARG


def test_an_adapter_workspace_serves_any_rank():
    for T, R in ((0, 8), (1, 8), (128, 16), (4000, 64)):
        n = moe.alloc_adapter_workspace(T, R, device="cpu").numel()
        assert n >= moe.moe_adapter_workspace_size(T, R) and n >= moe.moe_adapter_workspace_size(128, 128)
    with pytest.raises(moe.MoeError):
        moe.alloc_adapter_workspace(4, 12, device="cpu")

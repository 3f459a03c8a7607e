"""The MXFP4 and gated operators without a GPU: refusals, workspace sizes, and the plain forms
that the GPU tests compare with, pinned on hand-made cases."""
import ctypes

import numpy as np
import pytest
import torch

import plain_mx
import sparse_expert_ffn_route_gb300 as moe
from sparse_expert_ffn_route_gb300 import build as moe_build

FAKE = 1 << 20   # aligned, never dereferenced: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load_library()


def test_plain_quantizer_on_hand_made_blocks():
    x = np.zeros((1, 96))
    x[0, :8] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0]     # amax 5: e = 0; every tie
    x[0, 32:36] = [7.9, 6.5, -0.2, 0.3]                         # above 6 is held as 6
    x[0, 70] = np.inf
    code, scale = plain_mx.quantize(x)
    assert scale.tolist() == [[127, 127, 255]]
    assert code[0, :8].tolist() == [6, 0, 2, 2, 4, 4, 6, 14]
    assert code[0, 32:36].tolist() == [7, 7, 8, 1]
    assert not code[0, 64:].any() and np.isnan(plain_mx.values(code, scale)[0, 64:]).all()
    z = plain_mx.quantize(np.zeros((2, 32)))
    assert not z[0].any() and not z[1].any()
    p = plain_mx.pack(code)
    assert (plain_mx.unpack(p) == code).all() and p[0, 0] == 0x06 and p[0, 3] == 0xE6


def test_plain_slack_covers_what_lies_between():
    rng = np.random.default_rng(3)
    h = rng.standard_normal((40, 64))
    eh = np.full_like(h, 1e-3)
    slack = plain_mx.quantize_slack(h, eh)
    for _ in range(20):
        near = h + rng.uniform(-1, 1, h.shape) * eh
        assert (np.abs(plain_mx.held(near) - plain_mx.held(h)) <= slack + 1e-12).all()
    assert (slack == 0).mean() > 0.9


def test_quantize_refusals(lib):
    q = lib.moe_quantize_mxfp4
    ok = [FAKE, moe.MOE_DTYPE_F32, 64, 4, 64, FAKE, FAKE, None]

    def but(i, v):
        return q(*[v if k == i else a for k, a in enumerate(ok)])
    assert but(0, None) == moe.MOE_ERR_ARG and but(0, FAKE + 4) == moe.MOE_ERR_ALIGN
    assert but(1, 3) == moe.MOE_ERR_ARG and but(1, -1) == moe.MOE_ERR_ARG
    assert but(2, 63) == moe.MOE_ERR_SHAPE and but(2, 66) == moe.MOE_ERR_ALIGN
    assert but(3, -1) == moe.MOE_ERR_SHAPE and but(3, (1 << 27) + 1) == moe.MOE_ERR_SHAPE
    assert but(4, 48) == moe.MOE_ERR_SHAPE and but(4, 0) == moe.MOE_ERR_SHAPE
    assert but(5, None) == moe.MOE_ERR_ARG and but(6, FAKE + 8) == moe.MOE_ERR_ALIGN
    assert but(3, 0) == moe.MOE_OK     # nothing to do
    d = lib.moe_dequantize_mxfp4
    assert d(None, FAKE, 4, 64, FAKE, 0, None) == moe.MOE_ERR_ARG
    assert d(FAKE, FAKE, 4, 40, FAKE, 0, None) == moe.MOE_ERR_SHAPE
    assert d(FAKE, FAKE, 4, 64, FAKE + 2, 0, None) == moe.MOE_ERR_ALIGN
    assert d(FAKE, FAKE, 4, 64, FAKE, 7, None) == moe.MOE_ERR_ARG
    assert d(FAKE, FAKE, 0, 64, FAKE, 0, None) == moe.MOE_OK


def test_matmul_refusals(lib):
    ok = [FAKE, FAKE, 4, FAKE, FAKE, 2, FAKE, 100, 64, FAKE, 1, FAKE, 256, None]

    def but(i, v):
        return lib.moe_mxfp4_matmul(*[v if k == i else a for k, a in enumerate(ok)])
    for i in (0, 1, 3, 4, 9):
        assert but(i, None) == moe.MOE_ERR_ARG and but(i, FAKE + 8) == moe.MOE_ERR_ALIGN, i
    assert but(2, -1) == moe.MOE_ERR_SHAPE and but(2, 0) == moe.MOE_OK
    assert but(5, 0) == moe.MOE_ERR_SHAPE and but(5, 513) == moe.MOE_ERR_SHAPE
    assert but(6, None) == moe.MOE_ERR_ARG and but(6, FAKE + 2) == moe.MOE_ERR_ALIGN
    assert but(7, 0) == moe.MOE_ERR_SHAPE and but(8, 16) == moe.MOE_ERR_SHAPE
    assert but(10, 5) == moe.MOE_ERR_ARG
    assert but(11, None) == moe.MOE_ERR_WORKSPACE and but(11, FAKE + 16) == moe.MOE_ERR_ALIGN
    assert but(12, 255) == moe.MOE_ERR_WORKSPACE


def test_expert_ffn_refusals(lib):
    cfg = moe.MoeConfig.make(256, 8, 2, 128)
    one = moe.MoeConfig.make(256, 1, 1, 128)
    w = moe.ExpertMxfp4(*[FAKE] * 6)
    big = moe.moe_mxfp4_workspace_size(cfg, 4)

    def call(c=cfg, x=FAKE, dt=0, T=4, wt=w, off=FAKE, tok=FAKE, y=FAKE, ydt=0, ws=FAKE, n=big):
        return lib.moe_mxfp4_expert_ffn(ctypes.byref(c), x, dt, T, ctypes.byref(wt) if wt else None, off, tok, y,
                                        ydt, ws, n, None)
    assert call(x=None) == moe.MOE_ERR_ARG and call(x=FAKE + 4) == moe.MOE_ERR_ALIGN
    assert call(dt=9) == moe.MOE_ERR_ARG and call(ydt=9) == moe.MOE_ERR_ARG
    assert call(T=-1) == moe.MOE_ERR_SHAPE and call(T=0) == moe.MOE_OK
    assert call(wt=None) == moe.MOE_ERR_ARG
    assert call(wt=moe.ExpertMxfp4(*([FAKE] * 5 + [None]))) == moe.MOE_ERR_ARG
    assert "s_down" in moe.last_error()
    assert call(off=None) == moe.MOE_ERR_ARG and call(tok=None) == moe.MOE_ERR_ARG
    assert call(off=None, tok=None) == moe.MOE_ERR_ARG          # eight experts need a grouping
    assert call(off=FAKE + 2) == moe.MOE_ERR_ALIGN and call(y=None) == moe.MOE_ERR_ARG
    assert call(ws=None) == moe.MOE_ERR_WORKSPACE and call(n=big - 1) == moe.MOE_ERR_WORKSPACE
    assert call(c=moe.MoeConfig.make(100, 8, 2, 128)) == moe.MOE_ERR_SHAPE
    if not torch.cuda.is_available():
        assert call() == moe.MOE_ERR_UNSUPPORTED
        assert call(c=one, off=None, tok=None) == moe.MOE_ERR_UNSUPPORTED
    sizes = [moe.moe_mxfp4_workspace_size(cfg, t) for t in (0, 1, 16, 1000)]
    assert sizes[0] == 256 and sizes == sorted(sizes)
    assert moe.moe_mxfp4_workspace_size(cfg, -1) == 0
    assert moe.moe_mxfp4_workspace_size(moe.MoeConfig.make(100, 8, 2, 128), 4) == 0


def test_gated_refusals(lib):
    f_ok = [FAKE, 64, FAKE, FAKE, 1, 4, 64, 32, FAKE, FAKE, FAKE, FAKE, 256, None]

    def fwd(**kw):
        names = ("x", "ldx", "wg", "wu", "dt", "T", "H", "F", "h", "g", "u", "ws", "n", "st")
        return lib.moe_gated_forward(*[kw.get(k, v) for k, v in zip(names, f_ok)])
    for k in ("x", "wg", "wu", "h"):
        assert fwd(**{k: None}) == moe.MOE_ERR_ARG and fwd(**{k: FAKE + 8}) == moe.MOE_ERR_ALIGN, k
    assert fwd(g=None) == moe.MOE_ERR_ARG and fwd(u=FAKE + 2) == moe.MOE_ERR_ALIGN
    assert fwd(dt=moe.MOE_DTYPE_F32) == moe.MOE_ERR_ARG
    assert fwd(T=-1) == moe.MOE_ERR_SHAPE and fwd(T=0) == moe.MOE_OK
    assert fwd(H=60) == moe.MOE_ERR_SHAPE and fwd(F=0) == moe.MOE_ERR_SHAPE
    assert fwd(ldx=56) == moe.MOE_ERR_SHAPE and fwd(ldx=68) == moe.MOE_ERR_ALIGN
    assert fwd(ws=None) == moe.MOE_ERR_WORKSPACE and fwd(n=100) == moe.MOE_ERR_WORKSPACE
    need = moe.moe_gated_workspace_size(4, 64, 32, True)
    assert need > 256 and moe.moe_gated_workspace_size(4, 64, 32, False) == 256
    assert moe.moe_gated_workspace_size(4, 60, 32, True) == 0
    b_ok = [FAKE, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 1, 4, 64, 32, FAKE, FAKE, FAKE, FAKE, need, None]

    def bwd(**kw):
        names = ("dh", "x", "ldx", "wg", "wu", "g", "u", "dt", "T", "H", "F", "dx", "dwg", "dwu", "ws", "n", "st")
        return lib.moe_gated_backward(*[kw.get(k, v) for k, v in zip(names, b_ok)])
    for k in ("dh", "x", "wg", "wu", "g", "u"):
        assert bwd(**{k: None}) == moe.MOE_ERR_ARG, k
    assert bwd(dwg=None) == moe.MOE_ERR_ARG and bwd(dx=FAKE + 8) == moe.MOE_ERR_ALIGN
    assert bwd(n=need - 1) == moe.MOE_ERR_WORKSPACE
    assert bwd(T=0, dwg=None, dwu=None) == moe.MOE_OK


def test_binding_refuses_wrong_tensors(lib):
    x = torch.zeros(4, 64)
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_quantize_mxfp4(x, u8, u8[:, :2], stream=_NoStream)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        moe.moe_dequantize_mxfp4(u8, u8, x, stream=_NoStream)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        moe.moe_mxfp4_matmul(u8, u8[:, :2], u8, u8[:, :2], x, u8, stream=_NoStream)


class _NoStream:
    cuda_stream = 0

"""MXFP4 operators on the GPU against plain 64-bit forms (tests/plain_mx.py)."""
import numpy as np
import pytest
import torch

import plain_mx as pm
import sparse_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def random_mx(rng, *shape, spread=2):
    """Random codes and scales [..][K]: (codes, scales, packed codes, values)."""
    code = rng.integers(0, 16, shape).astype(np.uint8)
    scale = rng.integers(127 - spread, 128 + spread, shape[:-1] + (shape[-1] // 32,)).astype(np.uint8)
    return code, scale, pm.pack(code), pm.values(code, scale)


def quantize(x):
    codes = torch.full((*x.shape[:-1], x.shape[-1] // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((*x.shape[:-1], x.shape[-1] // 32), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4(x, codes, scales)
    return codes, scales


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 1120), (130, 2048), (1, 6144), (33, 1056)])
def test_quantize_is_exact(dtype, rows, K):
    rng = np.random.default_rng(rows * K)
    x = torch.from_numpy(rng.standard_normal((rows, K)) * np.exp(rng.standard_normal((rows, 1)))).to(dtype)
    x[rng.random((rows, K)) < 0.02] = 0
    x[0, :32] = 0
    codes, scales = quantize(x.cuda())
    code, scale = pm.quantize(x.double().numpy())
    assert (scales.cpu().numpy() == scale).all()
    assert (pm.unpack(codes.cpu().numpy()) == code).all()


def test_quantize_ties_extremes_and_nan():
    x = np.zeros((2, 12 * 32), np.float32)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0], np.float32)
    for i, s in enumerate((1.0, 2.0 ** -20, 2.0 ** 100)):
        x[0, 32 * i:32 * i + 8], x[0, 32 * i + 8:32 * i + 16] = ties * s, -ties * s
    x[0, 96:104] = np.finfo(np.float32).max                    # the largest finite number
    x[0, 128:136] = np.float32(1e-45) * np.arange(8)            # subnormal: e stays at -127
    x[0, 160:168] = np.float32(2.0 ** -126)
    x[0, 192], x[0, 224], x[0, 256], x[0, 257] = np.nan, np.inf, -np.inf, 1.0
    x[0, 288:320] = 7.999
    x[1] = x[0, ::-1]
    codes, scales = quantize(dev(x))
    code, scale = pm.quantize(x)
    assert (scales.cpu().numpy() == scale).all()
    assert (pm.unpack(codes.cpu().numpy()) == code).all()
    for dtype in TYPES:
        y = torch.empty(2, 12 * 32, dtype=dtype, device="cuda")
        moe.moe_dequantize_mxfp4(codes, scales, y)
        want = torch.from_numpy(pm.values(code, scale)).to(dtype)     # rounded once
        assert torch.equal(y.cpu().nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))


def test_quantize_strided_rows_and_more_dimensions():
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn(9, 256, generator=g, device="cuda")
    part = wide[:, 64:160]
    codes, scales = quantize(part.contiguous())
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    moe.moe_quantize_mxfp4(part, c2, s2)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    cube = torch.randn(2, 5, 64, generator=g, device="cuda")
    c3, s3 = quantize(cube)
    c4, s4 = quantize(cube.view(10, 64))
    assert torch.equal(c3.view(10, 32), c4) and torch.equal(s3.view(10, 2), s4)
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_mxfp4(wide[:, 3:99], c2, s2)             # rows off the 16-byte grid
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(wide.t(), c2, s2)


def matmul(px, sx, pw, sw, dtype, offsets=None, rows=None, fill=7.0):
    rows = px.shape[0]
    y = torch.full((rows, pw.shape[-2]), fill, dtype=dtype, device="cuda")
    ws = moe.alloc_mxfp4_matmul_workspace()
    moe.moe_mxfp4_matmul(dev(px), dev(sx), dev(pw), dev(sw), y, ws, offsets=None if offsets is None else dev(offsets))
    moe.moe_check_errors(ws)
    return y.cpu().double().numpy()


def check_matmul(got, vx, vw, dtype):
    """fp32 sums of K exact products, rounded once to the type."""
    want = vx @ vw.T
    bound = vx.shape[1] * pm.SUM * (np.abs(vx) @ np.abs(vw).T)
    assert (np.abs(got - want) <= bound * (1 + 2 ** -8) + pm.HALF_STEP[dtype] * np.abs(want) + 1e-30).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,N,K", [(1, 128, 256), (1, 1, 32), (5, 130, 96), (16, 64, 512), (17, 257, 1120),
                                      (33, 128, 160), (77, 1000, 1120), (192, 128, 256), (193, 300, 544),
                                      (400, 129, 2048), (24, 6144, 512), (25, 640, 512), (1, 512, 6144)])
def test_matmul(dtype, rows, N, K):
    rng = np.random.default_rng(rows + N + K)
    _, sx, px, vx = random_mx(rng, rows, K)
    _, sw, pw, vw = random_mx(rng, N, K)
    check_matmul(matmul(px, sx, pw, sw, dtype), vx, vw, dtype)


@pytest.mark.parametrize("counts", [[3, 0, 5], [0, 0, 0, 1], [40, 0, 1, 300, 7], [200, 200], [1] * 64, [0] * 9])
@pytest.mark.parametrize("N,K", [(130, 96), (256, 1024)])
def test_matmul_groups(counts, N, K):
    """Rows by group; rows outside every group keep what they had."""
    rng = np.random.default_rng(sum(counts) + N)
    before, after = 3, 2
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + before
    rows = int(off[-1]) + after
    _, sx, px, vx = random_mx(rng, rows, K)
    _, sw, pw, vw = random_mx(rng, len(counts), N, K)
    got = matmul(px, sx, pw, sw, torch.float32, offsets=off)
    assert (got[:before] == 7).all() and (got[rows - after:] == 7).all()
    for e in range(len(counts)):
        check_matmul(got[off[e]:off[e + 1]], vx[off[e]:off[e + 1]], vw[e], torch.float32)


def test_matmul_exact_in_small_integers():
    """Scales of one and short sums: every product and sum is exact."""
    rng = np.random.default_rng(0)
    code, _, px, _ = random_mx(rng, 50, 512)
    wcode, _, pw, _ = random_mx(rng, 200, 512)
    one = lambda n: np.full((n, 16), 127, np.uint8)  # noqa: E731
    got = matmul(px, one(50), pw, one(200), torch.float32)
    assert (got == pm.values(code, one(50)) @ pm.values(wcode, one(200)).T).all()


def test_matmul_each_input_and_scale_counts():
    """One nonzero input at a time: its code, its block's scale and its weight, and no other."""
    rng = np.random.default_rng(5)
    K, N = 608, 140
    wcode, sw, pw, vw = random_mx(rng, N, K, spread=6)
    code = np.zeros((K, K), np.uint8)
    code[np.arange(K), np.arange(K)] = 2           # 1.0
    scale = rng.integers(120, 135, (K, K // 32)).astype(np.uint8)
    got = matmul(pm.pack(code), scale, pw, sw, torch.float32)
    assert (got == pm.values(code, scale) @ vw.T).all()
    got = matmul(pm.pack(code[:16]), scale[:16], pw, sw, torch.float32)   # the few-row form
    assert (got == pm.values(code[:16], scale[:16]) @ vw.T).all()


def test_matmul_nan_blocks_stay_with_their_outputs():
    rng = np.random.default_rng(6)
    for rows in (9, 60):
        _, sx, px, vx = random_mx(rng, rows, 320)
        _, sw, pw, vw = random_mx(rng, 150, 320)
        sx[4, 3] = 255
        sw[17, 9] = 255
        got = matmul(px, sx, pw, sw, torch.float32)
        bad = np.zeros(got.shape, bool)
        bad[4], bad[:, 17] = True, True
        assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


def test_matmul_bad_offsets_are_recorded():
    rng = np.random.default_rng(7)
    _, sx, px, vx = random_mx(rng, 10, 64)
    _, sw, pw, vw = random_mx(rng, 3, 40, 64)
    for off, good in (([0, 4, 2, 10], [0, 2]), ([0, 4, 8, 11], [0, 1]), ([-1, 4, 8, 10], [1, 2])):
        y = torch.full((10, 40), 7.0, device="cuda")
        ws = moe.alloc_mxfp4_matmul_workspace()
        moe.moe_mxfp4_matmul(dev(px), dev(sx), dev(pw), dev(sw), y, ws, offsets=dev(np.array(off, np.int32)))
        with pytest.raises(moe.MoeError) as e:
            moe.moe_check_errors(ws)
        assert e.value.code == moe.MOE_ERR_DEVICE
        moe.moe_check_errors(ws)                     # reported once
        of = [[g for g in good if off[g] <= r < off[g + 1]] for r in range(10)]
        for r in range(10):
            if len(of[r]) == 1:      # a row that two groups claim holds either's result
                check_matmul(y.cpu().double().numpy()[r:r + 1], vx[r:r + 1], vw[of[r][0]], torch.float32)


def test_matmul_repeats_bit_for_bit_on_streams_and_in_graphs():
    rng = np.random.default_rng(8)
    _, sx, px, _ = random_mx(rng, 3, 2048)
    _, sw, pw, _ = random_mx(rng, 700, 2048)
    t = [dev(a) for a in (px, sx, pw, sw)]
    ws = moe.alloc_mxfp4_matmul_workspace()
    ys = [torch.empty(3, 700, device="cuda") for _ in range(3)]
    moe.moe_mxfp4_matmul(*t, ys[0], ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_mxfp4_matmul(*t, ys[1], ws, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_mxfp4_matmul(*t, ys[2], ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def expert_weights(rng, E, H, F):
    """Packed weights of E experts and their values, sized for outputs around one."""
    out, val = {}, {}
    for k, (n, kk) in {"gate": (F, H), "up": (F, H), "down": (H, F)}.items():
        code, scale, packed, _ = random_mx(rng, E, n, kk, spread=1)
        scale = (scale.astype(np.int64) - int(np.round(np.log2(2.93 * np.sqrt(kk))))).astype(np.uint8)
        out["w_" + k], out["s_" + k] = dev(packed), dev(scale)
        val[k] = pm.values(code, scale)
    return out, val


def check_ffn(got, x, val, e, dtype):
    """One expert's rows: h within its bound, requantised with the slack that leaves, then fp32
    sums of the down product and one rounding."""
    q = pm.held(x)
    _, _, h, eh, _, _ = pm.gate(q, val["gate"][e], val["up"][e])
    hq, slack, wd = pm.held(h), pm.quantize_slack(h, eh), val["down"][e]
    want = hq @ wd.T
    F = wd.shape[1]
    bound = slack @ np.abs(wd).T + F * pm.SUM * ((np.abs(hq) + slack) @ np.abs(wd).T)
    assert (np.abs(got - want) <= bound + pm.HALF_STEP[dtype] * (np.abs(want) + bound) + 1e-30).all()
    assert np.linalg.norm(got - want) <= 0.02 * np.linalg.norm(want) + 1e-30   # the slack is rarely used


@pytest.mark.parametrize("T,E,K,H,F", [(1, 8, 2, 256, 128), (5, 8, 2, 64, 64), (16, 8, 2, 256, 128), (40, 4, 4, 320, 192),
                                       (300, 8, 2, 256, 448), (700, 3, 2, 1088, 576), (1, 256, 8, 2048, 512)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_expert_ffn(T, E, K, H, F, dtype):
    rng = np.random.default_rng(T + E + H)
    cfg = moe.MoeConfig.make(H, E, K, F)
    w, val = expert_weights(rng, E, H, F)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dtype)
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)])
    if E > 2 and K < E:
        ids = np.where(ids == E - 1, (ids.max(1, keepdims=True) + 1) % E, ids)   # (often) an unused expert
        ids = np.stack([np.array(list(dict.fromkeys(r.tolist() + [e for e in range(E) if e not in r]))[:K]) for r in ids])
    order = np.argsort(ids.reshape(-1), kind="stable")
    tok = (order // K).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(ids.reshape(-1), minlength=E))]).astype(np.int32)
    y = torch.full((T * K, H), 7.0, device="cuda", dtype=dtype)
    ws = moe.alloc_mxfp4_workspace(cfg, T)
    moe.moe_mxfp4_expert_ffn(cfg, x.cuda(), w, y, ws, offsets=dev(off), tok=dev(tok))
    moe.moe_check_errors(ws)
    got, xd = y.cpu().double().numpy(), x.double().numpy()
    for e in range(E):
        if off[e] < off[e + 1]:
            check_ffn(got[off[e]:off[e + 1]], xd[tok[off[e]:off[e + 1]]], val, e, dtype)


def test_expert_ffn_dense_and_partial_lists():
    """One expert without lists; and lists shorter than the buffers (a keff below top_k)."""
    rng = np.random.default_rng(11)
    H, F = 192, 128
    w, val = expert_weights(rng, 1, H, F)
    x = rng.standard_normal((37, H)).astype(np.float32)
    one = moe.MoeConfig.make(H, 1, 1, F)
    y = torch.empty(37, H, device="cuda")
    ws = moe.alloc_mxfp4_workspace(one, 37)
    moe.moe_mxfp4_expert_ffn(one, dev(x), w, y, ws)
    moe.moe_check_errors(ws)
    check_ffn(y.cpu().double().numpy(), x.astype(np.float64), val, 0, torch.float32)

    cfg = moe.MoeConfig.make(H, 3, 2, F)
    w, val = expert_weights(rng, 3, H, F)
    off, tok = np.array([0, 2, 2, 3], np.int32), np.array([4, 0, 4] + [99999] * 7, np.int32)
    y = torch.full((10, H), 7.0, device="cuda")
    ws = moe.alloc_mxfp4_workspace(cfg, 5)
    moe.moe_mxfp4_expert_ffn(cfg, dev(x[:5]), w, y, ws, offsets=dev(off), tok=dev(tok))
    moe.moe_check_errors(ws)                                     # indices past the lists are not read
    got = y.cpu().double().numpy()
    check_ffn(got[:2], x[[4, 0]].astype(np.float64), val, 0, torch.float32)
    check_ffn(got[2:3], x[[4]].astype(np.float64), val, 2, torch.float32)
    assert (got[3:] == 7).all()


def test_expert_ffn_quantised_once_a_token():
    """Enough pairs that each token is quantised once and its row copied: lists that leave rows and
    an expert out, a bad index and a NaN row."""
    rng = np.random.default_rng(21)
    T, E, K, H, F = 1100, 4, 4, 2048, 64
    cfg = moe.MoeConfig.make(H, E, K, F)
    w, val = expert_weights(rng, E, H, F)
    x = rng.standard_normal((T, H)).astype(np.float32)
    x[7, 100] = np.inf
    counts = [900, 0, 1100, 300]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    tok = np.concatenate([rng.permutation(T)[:n] for n in counts] + [np.zeros(T * K - off[-1])]).astype(np.int32)
    tok[5] = T
    y = torch.full((T * K, H), 7.0, device="cuda")
    ws = moe.alloc_mxfp4_workspace(cfg, T)
    moe.moe_mxfp4_expert_ffn(cfg, dev(x), w, y, ws, offsets=dev(off), tok=dev(tok))
    with pytest.raises(moe.MoeError) as e:
        moe.moe_check_errors(ws)
    assert e.value.code == moe.MOE_ERR_DEVICE
    got = y.cpu().double().numpy()
    assert (got[off[-1]:] == 7).all()
    nan = np.zeros(T * K, bool)
    nan[:off[-1]] = (tok[:off[-1]] == 7) | (tok[:off[-1]] == T)
    assert np.isnan(got[nan]).all() and np.isfinite(got[~nan]).all()
    for e in range(E):
        rows = np.arange(off[e], off[e + 1])
        rows = rows[~nan[rows]]
        if len(rows):
            check_ffn(got[rows], x[tok[rows]].astype(np.float64), val, e, torch.float32)


def test_expert_ffn_bad_token_and_nan_rows():
    rng = np.random.default_rng(12)
    H, F = 128, 64
    cfg = moe.MoeConfig.make(H, 2, 1, F)
    w, val = expert_weights(rng, 2, H, F)
    x = rng.standard_normal((4, H)).astype(np.float32)
    x[2, 5] = np.nan
    off, tok = np.array([0, 2, 4], np.int32), np.array([0, 4, 2, 3], np.int32)   # 4 is no token
    y = torch.zeros(4, H, device="cuda")
    ws = moe.alloc_mxfp4_workspace(cfg, 4)
    moe.moe_mxfp4_expert_ffn(cfg, dev(x), w, y, ws, offsets=dev(off), tok=dev(tok))
    with pytest.raises(moe.MoeError) as e:
        moe.moe_check_errors(ws)
    assert e.value.code == moe.MOE_ERR_DEVICE
    got = y.cpu().double().numpy()
    assert np.isnan(got[1]).all() and np.isnan(got[2]).all()
    check_ffn(got[:1], x[:1].astype(np.float64), val, 0, torch.float32)
    check_ffn(got[3:], x[3:].astype(np.float64), val, 1, torch.float32)


def test_routed_layer_on_mxfp4_experts():
    """route -> permute -> MXFP4 experts -> combine, with a shared expert through the dense form."""
    rng = np.random.default_rng(13)
    T, H, E, K, F = 21, 256, 8, 2, 128
    cfg = moe.MoeConfig.make(H, E, K, F)
    one = moe.MoeConfig.make(H, 1, 1, F)
    w, val = expert_weights(rng, E, H, F)
    sw, sval = expert_weights(rng, 1, H, F)
    x = rng.standard_normal((T, H)).astype(np.float32)
    xd, wr = dev(x), dev((rng.standard_normal((E, H)) / 16).astype(np.float32))
    ws, ms = moe.alloc_workspace(cfg, T), moe.alloc_mxfp4_workspace(cfg, T)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, keff, wt = i32(T, K), i32(T), torch.empty(T, K, device="cuda")
    counts, off, tok, slot, uniq, nu = i32(E), i32(E + 1), i32(T * K), i32(T * K), i32(E), i32(1)
    moe.moe_route(cfg, xd, wr, torch.zeros(E, device="cuda"), ids, wt, keff, ws)
    moe.moe_permute(cfg, ids, keff, counts, off, tok, slot, uniq, nu, ws)
    yp, y, ysh = torch.empty(T * K, H, device="cuda"), torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    moe.moe_mxfp4_expert_ffn(cfg, xd, w, yp, ms, offsets=off, tok=tok)
    moe.moe_mxfp4_expert_ffn(one, xd, sw, ysh, ms)
    moe.moe_combine(cfg, yp, ids, keff, wt, off, tok, y, ws)
    y += ysh
    moe.moe_check_errors(ws)
    moe.moe_check_errors(ms)
    want = np.zeros((T, H))
    q = pm.held(x.astype(np.float64))
    for t in range(T):
        want[t] = pm.held(pm.gate(q[t:t + 1], sval["gate"][0], sval["up"][0])[2])[0] @ sval["down"][0].T
        for k in range(K):
            e = int(ids[t, k])
            want[t] += float(wt[t, k]) * (pm.held(pm.gate(q[t:t + 1], val["gate"][e], val["up"][e])[2])[0] @ val["down"][e].T)
    assert np.linalg.norm(y.cpu().double().numpy() - want) <= 0.02 * np.linalg.norm(want)


@pytest.mark.parametrize("rows,N,K", [(300, 1500, 2048), (2048, 2100, 512), (1000, 4000, 96), (900, 513, 1120)])
def test_matmul_large_tiles(rows, N, K):
    """Sizes at which tiles hold 256 and 512 weight rows, with ragged last tiles of either side."""
    rng = np.random.default_rng(rows + N)
    _, sx, px, vx = random_mx(rng, rows, K)
    _, sw, pw, vw = random_mx(rng, N, K)
    check_matmul(matmul(px, sx, pw, sw, torch.bfloat16), vx, vw, torch.bfloat16)

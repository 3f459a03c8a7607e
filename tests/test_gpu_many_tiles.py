"""Sizes at which the tensor-core kernels of the MXFP4 operators and the gated block run more than
one tile on a CTA or a pair of SMs, and the tiles of 512 weight rows: the forms that large calls
take.  Against plain forms in 64 bits (on the GPU, by library products)."""
import numpy as np
import pytest
import torch

import plain_mx as pm
import sparse_expert_ffn_route_gb300 as moe
from test_gpu_gated import subnormal
from test_gpu_mxfp4 import check_ffn, dev, expert_weights

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def tiles(rows, cols, groups=1):
    """The fewest tiles (256 rows x at most 256 columns) that a product of the gated block takes."""
    return groups * -(-rows // 256) * -(-cols // 256)


def make(T, H, F, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return rand(T, H).to(dtype), (rand(F, H) / H ** 0.5).to(dtype), (rand(F, H) / H ** 0.5).to(dtype), rand(T, F).to(dtype)


def step(x, wg, wu, dh, out, ws):
    h, g, u, dx, dwg, dwu = out
    moe.moe_gated_forward(x, wg, wu, h, ws, g=g, u=u)
    moe.moe_gated_backward(dh, x, wg, wu, g, u, dx, dwg, dwu, ws)


def buffers(T, H, F, dtype):
    return [torch.full(s, 7.0, dtype=dtype, device="cuda") for s in ((T, F), (T, F), (T, F), (T, H), (F, H), (F, H))]


def check_step(x, wg, wu, dh, out):
    """Every rounding at its worst: fp32 sums; h one rounding; of each factor of dh at most half a
    step of the larger one; dg, du and the gradients one rounding each."""
    dtype = x.dtype
    r, z = pm.HALF_STEP[dtype], subnormal(dtype)
    X, WG, WU, DH = (t.double() for t in (x, wg, wu, dh))
    G, U = X @ WG.T, X @ WU.T
    K = X.shape[1]
    eg, eu = K * pm.SUM * (X.abs() @ WG.abs().T), K * pm.SUM * (X.abs() @ WU.abs().T)
    s = torch.sigmoid(G)
    A, B, e32 = U * s * (1 + G * (1 - s)), G * s, 10 * 2.0 ** -24

    def close(got, want, bound):
        assert ((got.double() - want).abs() <= bound * (1 + r) + r * want.abs() + z).all()
    close(out[0], B * U, 1.1 * eg * (U.abs() + eu) + B.abs() * eu + e32 * (B * U).abs())
    kept = r * torch.maximum(A.abs(), B.abs()) + z
    eA = 1.1 * eu + 0.5 * (U.abs() + eu) * eg + e32 * U.abs() * s * (1 + G.abs() * (1 + s)) + kept
    eB = 1.1 * eg + e32 * B.abs() + kept
    dg, du = DH * A, DH * B
    edg, edu = DH.abs() * eA * (1 + r) + r * dg.abs() + z, DH.abs() * eB * (1 + r) + r * du.abs() + z

    def product(got, pairs):
        n = sum(a.shape[1] for a, _, _ in pairs)
        bound = sum(e @ b.abs() for _, b, e in pairs) + n * pm.SUM * sum((a.abs() + e) @ b.abs() for a, b, e in pairs)
        close(got, sum(a @ b for a, b, _ in pairs), bound)
    product(out[3], [(dg, WG, edg), (du, WU, edu)])
    product(out[4], [(dg.T, X, edg.T)])
    product(out[5], [(du.T, X, edu.T)])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,F", [(2100, 2056, 2056), (4100, 72, 4104), (4100, 4104, 72)])
def test_gated_step_of_several_waves(dtype, T, H, F):
    """Two waves of pairs and more, the last tile of rows and of columns ragged: in all three products
    of the first size, in the forward pass and in dx of the others."""
    pairs = sms() // 2
    assert max(tiles(T, F), tiles(T, H)) > pairs and (H == 72 or F == 72 or min(tiles(T, F), tiles(T, H), tiles(F, H, 2)) > pairs)
    t = make(T, H, F, dtype)
    out, ws = buffers(T, H, F, dtype), moe.alloc_gated_workspace(T, H, F, True)
    step(*t, out, ws)
    moe.moe_check_errors(ws)
    check_step(*t, out)


def test_gated_steps_back_to_back():
    """Steps of three sets of inputs in turn, with nothing between them: each time the same bits as
    the set's first step."""
    T, H, F = 2100, 2056, 2056
    sets = [(make(T, H, F, torch.bfloat16, seed), buffers(T, H, F, torch.bfloat16), moe.alloc_gated_workspace(T, H, F, True))
            for seed in range(3)]
    first = []
    for t, out, ws in sets:
        step(*t, out, ws)
        first.append([o.clone() for o in out])
    for _ in range(20):
        for t, out, ws in sets:
            step(*t, out, ws)
    for (_, out, ws), want in zip(sets, first):
        moe.moe_check_errors(ws)
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(out, want))


def values64(packed, scale):
    """MXFP4 codes and scales on the GPU -> 64-bit values."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    v = torch.stack([grid[(packed & 15).long()], grid[(packed >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(scale.double() - 127).repeat_interleave(32, -1)


def check_product(got, x, w, dtype):
    want = x @ w.T
    bound = x.shape[1] * pm.SUM * (x.abs() @ w.abs().T)
    assert ((got.double() - want).abs() <= bound * (1 + 2 ** -8) + pm.HALF_STEP[dtype] * want.abs() + 1e-30).all()


def random_gpu(g, *shape):
    packed = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device="cuda", dtype=torch.uint8)
    return packed, torch.randint(125, 130, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda", dtype=torch.uint8)


@pytest.mark.parametrize("rows,N,K", [(2100, 2500, 544), (2100, 2500, 512), (700, 4900, 2048), (697, 5000, 2080), (4096, 6144, 6144)])
def test_product_of_several_waves(rows, N, K):
    """Pairs with more than one tile, of 256 weight rows (first two) and of 512 (the others: the rule
    on the host takes them for long reductions over many rows; the last more than one a pair)."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    (px, sx), (pw, sw) = random_gpu(g, rows, K), random_gpu(g, N, K)
    y, ws = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda"), moe.alloc_mxfp4_matmul_workspace()
    for _ in range(3):
        moe.moe_mxfp4_matmul(px, sx, pw, sw, y, ws)
    moe.moe_check_errors(ws)
    check_product(y, values64(px, sx), values64(pw, sw), torch.bfloat16)


@pytest.mark.parametrize("K", [512, 544])
def test_product_of_few_rows_and_many_tiles(K):
    """More tiles of the few-row form than CTAs that are resident (two an SM)."""
    rng = np.random.default_rng(K)
    E, N = 72, 1000
    counts = rng.integers(0, 40, E)
    counts[::9] = 0
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1])
    assert rows <= 24 * E and 8 * (counts > 0).sum() > 2 * sms()
    g = torch.Generator(device="cuda").manual_seed(K)
    (px, sx), (pw, sw) = random_gpu(g, rows, K), random_gpu(g, E, N, K)
    y, ws = torch.full((rows, N), 7.0, dtype=torch.float32, device="cuda"), moe.alloc_mxfp4_matmul_workspace()
    for _ in range(3):
        moe.moe_mxfp4_matmul(px, sx, pw, sw, y, ws, offsets=dev(off))
    moe.moe_check_errors(ws)
    x, w = values64(px, sx), values64(pw, sw)
    for e in range(E):
        check_product(y[off[e]:off[e + 1]], x[off[e]:off[e + 1]], w[e], torch.float32)


def test_product_of_lists_that_name_rows_again():
    """Groups out of order are recorded and left out; the others here name every row five times, more
    tiles of the few-row form than the host counts on, so that a cluster which shares a tile's
    reduction takes a second one.  (All groups' weights are alike: it does not matter whose row it is.)"""
    g = torch.Generator(device="cuda").manual_seed(5)
    E, rows, N, K = 9, 64, 100, 4096
    (px, sx), (pw, sw) = random_gpu(g, rows, K), random_gpu(g, 1, N, K)
    off = torch.tensor([0, rows] * 5, dtype=torch.int32, device="cuda")
    y, ws = torch.full((rows, N), 7.0, dtype=torch.float32, device="cuda"), moe.alloc_mxfp4_matmul_workspace()
    moe.moe_mxfp4_matmul(px, sx, pw.repeat(E, 1, 1), sw.repeat(E, 1, 1), y, ws, offsets=off)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_check_errors(ws)
    assert e.value.code == moe.MOE_ERR_DEVICE          # the lists, and no wait that gave up
    check_product(y, values64(px, sx), values64(pw[0], sw[0]), torch.float32)


@pytest.mark.parametrize("counts,H,F", [([1500, 0, 1, 800, 299], 128, 1984), ([17, 24, 3, 0, 31, 22, 8, 1] * 10, 256, 960)])
def test_expert_ffn_of_many_tiles(counts, H, F):
    """The gate/up form on pairs with more tiles than pairs (first), and the few-row form with more
    tiles than resident CTAs (second)."""
    rng = np.random.default_rng(F)
    E, P = len(counts), sum(counts)
    few = P <= 24 * E
    ntiles = sum(-(-F // (128 if few else 256)) * -(-n // (32 if few else 224)) for n in counts)
    assert ntiles > (2 * sms() if few else sms() // 2)
    cfg = moe.MoeConfig.make(H, E, 1, F)
    w, val = expert_weights(rng, E, H, F)
    x = rng.standard_normal((P, H)).astype(np.float32)
    off, tok = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), rng.permutation(P).astype(np.int32)
    y, ws = torch.full((P, H), 7.0, device="cuda"), moe.alloc_mxfp4_workspace(cfg, P)
    xd, od, td = dev(x), dev(off), dev(tok)
    for _ in range(3):
        moe.moe_mxfp4_expert_ffn(cfg, xd, w, y, ws, offsets=od, tok=td)
    moe.moe_check_errors(ws)
    got = y.cpu().double().numpy()
    for e in range(E):
        if counts[e]:
            at = slice(off[e], off[e + 1])
            check_ffn(got[at], x[tok[at]].astype(np.float64), val, e, torch.float32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,F", [(16, 520, 20000), (64, 2056, 10008)])
def test_gated_forward_of_few_tokens_and_many_tiles(dtype, T, H, F):
    """More tiles of the few-token form than SMs."""
    assert -(-F // 128) * -(-T // 32) > sms()
    x, wg, wu, _ = make(T, H, F, dtype)
    h, ws = torch.full((T, F), 7.0, dtype=dtype, device="cuda"), moe.alloc_gated_workspace(T, H, F, False)
    for _ in range(3):
        moe.moe_gated_forward(x, wg, wu, h, ws)
    moe.moe_check_errors(ws)
    X, WG, WU = (t.double() for t in (x, wg, wu))
    G, U = X @ WG.T, X @ WU.T
    eg, eu = H * pm.SUM * (X.abs() @ WG.abs().T), H * pm.SUM * (X.abs() @ WU.abs().T)
    S = G * torch.sigmoid(G)
    r = pm.HALF_STEP[dtype]
    bound = 1.1 * eg * (U.abs() + eu) + S.abs() * eu + 8 * 2.0 ** -24 * (S * U).abs()
    assert ((h.double() - S * U).abs() <= bound * (1 + r) + r * (S * U).abs() + subnormal(dtype)).all()

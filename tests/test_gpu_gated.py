"""The 16-bit gated block and its gradients on the GPU against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import plain_mx as pm
import sparse_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]
SIZES = [(1, 64, 64), (1, 1000, 520), (2, 8, 8), (16, 256, 136), (32, 6144, 256), (33, 264, 128), (70, 136, 1000),
         (256, 128, 256), (300, 520, 264), (513, 72, 328), (50, 2048, 136), (17, 1032, 72),
         (64, 2056, 392)]


def make(T, H, F, dtype, seed=0):
    rng = np.random.default_rng(seed + T + H + F)
    t = lambda *s, c=1.0: torch.from_numpy(rng.standard_normal(s) * c).to(dtype)  # noqa: E731
    return t(T, H), t(F, H, c=H ** -0.5), t(F, H, c=H ** -0.5), t(T, F)


def forward(x, wg, wu, keep=True):
    T, F = x.shape[0], wg.shape[0]
    b = [torch.full((T, F), 7.0, dtype=x.dtype, device="cuda") for _ in range(3)]
    ws = moe.alloc_gated_workspace(T, x.shape[1], F, True)
    moe.moe_gated_forward(x, wg, wu, b[0], ws, g=b[1] if keep else None, u=b[2] if keep else None)
    moe.moe_check_errors(ws)
    return b


def f64(t):
    return t.detach().cpu().double().numpy()


def subnormal(dtype):
    """Half the spacing of the type's subnormal numbers: the least error of a rounding."""
    return float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps / 2


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,F", SIZES)
def test_forward(dtype, T, H, F):
    x, wg, wu, _ = make(T, H, F, dtype)
    h = f64(forward(x.cuda(), wg.cuda(), wu.cuda())[0])
    _, _, want, bound, _, _ = pm.gate(f64(x), f64(wg), f64(wu))
    r, z = pm.HALF_STEP[dtype], subnormal(dtype)
    assert (np.abs(h - want) <= bound + r * (np.abs(want) + bound) + z).all()
    h2 = f64(forward(x.cuda(), wg.cuda(), wu.cuda(), keep=False)[0])
    assert (h2 == h).all()


def backward(dh, x, wg, wu, g, u):
    T, H = x.shape
    F = wg.shape[0]
    out = [torch.full(s, 7.0, dtype=x.dtype, device="cuda") for s in ((T, H), (F, H), (F, H))]
    ws = moe.alloc_gated_workspace(T, H, F, True)
    moe.moe_gated_backward(dh, x, wg, wu, g, u, *out, ws)
    moe.moe_check_errors(ws)
    return out


# what one kept factor is off by at most, relative to the larger of the element's two, and absolutely
KEPT = {torch.bfloat16: 1 / 2047, torch.float16: 1 / 5792}
KEPT_LEAST = {torch.bfloat16: 2.0 ** -103 * 2 / 2047, torch.float16: 2.0 ** -13 * 2 / 5792}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,F", SIZES)
def test_backward(dtype, T, H, F):
    """The factors A = u s (1 + g (1 - s)) and B = g s of fp32 sums, 10 fp32 roundings and the kept
    form's step; dg and du one rounding to the type, the products fp32 sums, the gradients one
    rounding."""
    x, wg, wu, dh = make(T, H, F, dtype)
    _, g, u = forward(x.cuda(), wg.cuda(), wu.cuda())
    dx, dwg, dwu = (f64(t) for t in backward(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), g, u))
    X, WG, WU, DH = (f64(t) for t in (x, wg, wu, dh))
    G, U, _, _, eg, eu = pm.gate(X, WG, WU)
    s = pm.sigmoid(G)
    r, z = pm.HALF_STEP[dtype], subnormal(dtype)
    A, B = U * s * (1 + G * (1 - s)), G * s
    e32 = 10 * 2.0 ** -24
    # |silu'| <= 1.1 and |silu''| <= 0.5; 1 + g (1 - s) is a sum: its roundings are relative to its terms
    kept = KEPT[dtype] * np.maximum(np.abs(A), np.abs(B)) + KEPT_LEAST[dtype]
    eA = 1.1 * eu + 0.5 * (np.abs(U) + eu) * eg + e32 * np.abs(U) * s * (1 + np.abs(G) * (1 + s))
    eB = 1.1 * eg + e32 * np.abs(B)
    eA, eB = eA + kept + KEPT[dtype] * (eA + eB), eB + kept + KEPT[dtype] * (eA + eB)
    dg, du = DH * A, DH * B
    edg = np.abs(DH) * eA * (1 + r) + r * np.abs(dg) + z
    edu = np.abs(DH) * eB * (1 + r) + r * np.abs(du) + z

    def check(got, pairs):
        want = sum(a @ b for a, b, _ in pairs)
        mags = sum((np.abs(a) + e) @ np.abs(b) for a, b, e in pairs)
        n = sum(a.shape[1] for a, _, _ in pairs)
        bound = sum(e @ np.abs(b) for _, b, e in pairs) + n * pm.SUM * mags
        assert (np.abs(got - want) <= bound * (1 + r) + r * np.abs(want) + z).all()
    check(dx, [(dg, WG, edg), (du, WU, edu)])
    check(dwg, [(dg.T, X, edg.T)])
    check(dwu, [(du.T, X, edu.T)])


def test_gradient_against_differences():
    """d/de of sum(h(x + e a, Wg + e b, Wu + e c) * dh) in 64 bits, by central differences, against
    the gradients' inner products with a, b, c."""
    T, H, F = 40, 128, 96
    x, wg, wu, dh = make(T, H, F, torch.float16, seed=5)
    _, g, u = forward(x.cuda(), wg.cuda(), wu.cuda())
    dx, dwg, dwu = (f64(t) for t in backward(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), g, u))
    X, WG, WU, DH = (f64(t) for t in (x, wg, wu, dh))
    rng = np.random.default_rng(9)

    def loss(a, b, c):
        p = a @ b.T
        return (p * pm.sigmoid(p) * (a @ c.T) * DH).sum()
    for grad, at in ((dx, 0), (dwg, 1), (dwu, 2)):
        a = rng.standard_normal(grad.shape)
        d = [np.zeros_like(v) for v in (X, WG, WU)]
        d[at] = a
        e = 1e-5
        want = (loss(X + e * d[0], WG + e * d[1], WU + e * d[2]) - loss(X - e * d[0], WG - e * d[1], WU - e * d[2])) / (2 * e)
        # two roundings to fp16 (dg or du, the gradient) and the kept factors' step, each at most
        # half a step of its value: sum over the entries in the worst case is far above; in the
        # mean of n independent entries it is the norm's
        bound = 5 * pm.HALF_STEP[torch.float16] * np.linalg.norm(grad) * 6 + 1e-6 * abs(want)
        assert abs((grad * a).sum() - want) <= bound


def same(a, b):
    """The same bits (what the forward pass keeps is words, not numbers of the type)."""
    return all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(a, b))


def test_strided_rows_of_x():
    x, wg, wu, dh = (t.cuda() for t in make(50, 128, 64, torch.bfloat16))
    wide = torch.full((50, 200), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 24:152] = x
    part = wide[:, 24:152]
    a, b = forward(x, wg, wu), forward(part, wg, wu)
    assert same(a, b)
    ga, gb = backward(dh, x, wg, wu, a[1], a[2]), backward(dh, part, wg, wu, a[1], a[2])
    assert same(ga, gb)


def test_each_gradient_alone_and_repeats():
    x, wg, wu, dh = (t.cuda() for t in make(65, 264, 136, torch.bfloat16))
    _, g, u = forward(x, wg, wu)
    dx, dwg, dwu = backward(dh, x, wg, wu, g, u)
    ws = moe.alloc_gated_workspace(65, 264, 136, True)
    dx2, dwg2, dwu2 = torch.empty_like(dx), torch.empty_like(dwg), torch.empty_like(dwu)
    moe.moe_gated_backward(dh, x, wg, wu, g, u, dx2, None, None, ws)
    moe.moe_gated_backward(dh, x, wg, wu, g, u, None, dwg2, dwu2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dwg, dwg2) and torch.equal(dwu, dwu2)


def test_no_rows():
    x, wg, wu, dh = (t.cuda() for t in make(1, 64, 32, torch.bfloat16))
    e, h = x[:0], dh[:0]
    ws = moe.alloc_gated_workspace(1, 64, 32, True)
    moe.moe_gated_forward(e, wg, wu, h, ws)
    dwg, dwu = torch.full_like(wg, 7.0), torch.full_like(wu, 7.0)
    moe.moe_gated_backward(h, e, wg, wu, h, h, e, dwg, dwu, ws)
    assert not dwg.any() and not dwu.any()


def test_saturated_gates_and_infinities():
    """Large |g| (sigmoid 0 or 1, exp overflow) stays finite; an infinite input stays in its row."""
    T, H, F = 40, 64, 64
    x, wg, wu, dh = make(T, H, F, torch.bfloat16)
    big = (x * 200).cuda()
    h, g, u = forward(big, wg.cuda(), wu.cuda())
    assert torch.isfinite(h).all()
    out = backward(dh.cuda(), big, wg.cuda(), wu.cuda(), g, u)
    assert all(torch.isfinite(t).all() for t in out)
    x[3, 5] = float("inf")
    h = forward(x.cuda(), wg.cuda(), wu.cuda())[0]
    rows = torch.isfinite(h).all(1)
    assert not rows[3] and rows.sum() == T - 1


def test_step_in_a_graph():
    x, wg, wu, dh = (t.cuda() for t in make(90, 256, 128, torch.bfloat16))
    want = forward(x, wg, wu)
    grads = backward(dh, x, wg, wu, want[1], want[2])
    ws = moe.alloc_gated_workspace(90, 256, 128, True)
    b = [torch.zeros_like(t) for t in want]
    o = [torch.zeros_like(t) for t in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_gated_forward(x, wg, wu, b[0], ws, g=b[1], u=b[2])
        moe.moe_gated_backward(dh, x, wg, wu, b[1], b[2], *o, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    moe.moe_check_errors(ws)
    assert same(want + grads, b + o)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.0, 1e-6, 1e-3, 1.0, 30.0])
def test_kept_factors_over_the_range(dtype, scale):
    """One input and identity-like weights: g and u are chosen freely, dh = 1, x' = 1, so that dwg and
    dwu are the rounded factors themselves, down to the least kept step and at zero."""
    F = 256
    rng = np.random.default_rng(17)
    x = torch.zeros(1, 8, dtype=dtype)
    x[0, 0] = 1
    wg, wu = torch.zeros(F, 8, dtype=dtype), torch.zeros(F, 8, dtype=dtype)
    wg[:, 0] = torch.from_numpy(rng.standard_normal(F) * min(scale, 5.0)).to(dtype)
    wu[:, 0] = torch.from_numpy(rng.standard_normal(F) * scale * 10.0 ** rng.uniform(-3, 0, F)).to(dtype)
    dh = torch.ones(1, F, dtype=dtype)
    _, g, u = forward(x.cuda(), wg.cuda(), wu.cuda())
    _, dwg, dwu = (f64(t) for t in backward(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), g, u))
    G, U = f64(wg)[:, 0], f64(wu)[:, 0]
    s = pm.sigmoid(G)
    A, B = U * s * (1 + G * (1 - s)), G * s
    kept = KEPT[dtype] * np.maximum(np.abs(A), np.abs(B)) + KEPT_LEAST[dtype] + 10 * 2.0 ** -24 * np.maximum(np.abs(U), np.abs(G)) * (1 + np.abs(G))
    r, z = pm.HALF_STEP[dtype], subnormal(dtype)
    for got, want in ((dwg[:, 0], A), (dwu[:, 0], B)):
        # the rounding to dg or du, then the gradient's (of a value that the type holds: none)
        assert (np.abs(got - want) <= kept * (1 + r) + r * np.abs(want) + z).all()


def test_factors_that_are_not_finite():
    """An infinite g or u makes its row's dg and du NaN and no other row's."""
    x, wg, wu, dh = make(40, 64, 64, torch.bfloat16)
    x[3, 5] = float("inf")
    _, g, u = forward(x.cuda(), wg.cuda(), wu.cuda())
    dx = backward(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), g, u)[0]
    rows = torch.isfinite(dx).all(1)
    assert not rows[3] and rows.sum() == 39

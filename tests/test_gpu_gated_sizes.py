"""Gradients of the gated block where g and u differ in size: each gradient against 64 bits by the size
of its own terms, whatever the other factor's."""
import numpy as np
import pytest
import torch

import plain_mx as pm
import sparse_expert_ffn_route_gb300 as moe
from test_gpu_gated import backward, f64, forward, make, subnormal

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]
# standard deviations of g and u
SIZES = [(1, 1), (0.1, 10), (1, 0.01), (1, 0.001), (1, 1e-4), (1, 100), (0.01, 1), (0.001, 1), (5, 1)]


def kept(v, dtype):
    """What a kept factor of value v is off by at most."""
    if dtype == torch.float16:
        return 2.0 ** -11 * np.abs(v) + 2.0 ** -25
    a = np.abs(v)
    return np.where((a > 2.0 ** -12) & (a < 16), 2.0 ** -11, 2.0 ** -8) * a * (1 + 2.0 ** -8) + 2.0 ** -84


def parts(X, WG, WU, DH, dtype):
    """The 64-bit gradients with what bounds them: for each, pairs (factor, its largest error, matrix)."""
    G, U, _, _, eg, eu = pm.gate(X, WG, WU)
    s = pm.sigmoid(G)
    r, z, e32 = pm.HALF_STEP[dtype], subnormal(dtype), 10 * 2.0 ** -24
    A, B = U * s * (1 + G * (1 - s)), G * s
    # |silu'| <= 1.1 and |silu''| <= 0.5; 1 + g (1 - s) is a sum: its roundings are relative to its terms
    eA = 1.1 * eu + 0.5 * (np.abs(U) + eu) * eg + e32 * np.abs(U) * s * (1 + np.abs(G) * (1 + s))
    eB = 1.1 * eg + e32 * np.abs(B)
    out = []
    for v, e in ((A, eA), (B, eB)):
        e = e + kept(np.abs(v) + e, dtype)
        out.append((DH * v, np.abs(DH) * e * (1 + r) + r * np.abs(DH * v) + z, np.abs(DH) * kept(v, dtype)))
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sg,su", SIZES)
def test_gradients_by_their_own_size(dtype, sg, su):
    """Element by element with every rounding at its worst, and in the norm, where independent roundings
    of at most half a step add as squares (a uniform error's square is a third of its largest)."""
    T, H, F = 512, 256, 256
    x, wg, wu, dh = make(T, H, F, dtype, seed=3)
    wg, wu = (wg.double() * sg).to(dtype), (wu.double() * su).to(dtype)
    _, g, u = forward(x.cuda(), wg.cuda(), wu.cuda())
    dx, dwg, dwu = (f64(t) for t in backward(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), g, u))
    X, WG, WU, DH = (f64(t) for t in (x, wg, wu, dh))
    r, z = pm.HALF_STEP[dtype], subnormal(dtype)
    (dg, edg, kdg), (du, edu, kdu) = parts(X, WG, WU, DH, dtype)

    def check(got, pairs):
        want = sum(a @ b for a, _, _, b in pairs)
        n = sum(a.shape[1] for a, _, _, _ in pairs)
        sums = n * pm.SUM * sum((np.abs(a) + e) @ np.abs(b) for a, e, _, b in pairs)
        bound = sum(e @ np.abs(b) for _, e, _, b in pairs) + sums
        off = np.abs(got - want)
        assert (off <= bound * (1 + r) + r * np.abs(want) + z).all()
        square = sum(((r * a) ** 2 + k ** 2 + z ** 2) @ b ** 2 for a, _, k, b in pairs).sum() + ((r * want) ** 2 + z ** 2).sum()
        # 5 % for the fluctuation of tens of thousands of errors; fp32 roundings are far below
        assert np.linalg.norm(off) <= 1.05 * np.sqrt(square / 3)
    check(dx, [(dg, edg, kdg, WG), (du, edu, kdu, WU)])
    check(dwg, [(dg.T, edg.T, kdg.T, X)])
    check(dwu, [(du.T, edu.T, kdu.T, X)])


@pytest.mark.parametrize("sg,su", [(1, 1), (1, 0.001), (0.001, 1), (1, 30)])
def test_gradients_against_differences(sg, su):
    """Inner products with random directions against central differences in 64 bits.  The gradient's error
    is within a half step of its norm (three roundings of it, as squares), its product with a direction
    of independent entries normal of that size: five times it."""
    dtype, T, H, F = torch.float16, 40, 128, 96
    x, wg, wu, dh = make(T, H, F, dtype, seed=5)
    wg, wu = (wg.double() * sg).to(dtype), (wu.double() * su).to(dtype)
    _, g, u = forward(x.cuda(), wg.cuda(), wu.cuda())
    grads = [f64(t) for t in backward(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), g, u)]
    at = [f64(t) for t in (x, wg, wu)]
    DH = f64(dh)
    rng = np.random.default_rng(11)

    def loss(a, b, c):
        p = a @ b.T
        return (p * pm.sigmoid(p) * (a @ c.T) * DH).sum()
    for i, grad in enumerate(grads):
        for _ in range(4):
            d = rng.standard_normal(grad.shape)
            e = 1e-5
            lo, hi = [v.copy() for v in at], [v.copy() for v in at]
            lo[i] -= e * d
            hi[i] += e * d
            want = (loss(*hi) - loss(*lo)) / (2 * e)
            # the differences' own error: a few ulp of the loss over the step
            own = 64 * 2.0 ** -52 * np.abs(loss(*at)) / e + 1e-7 * abs(want)
            small = 2.0 ** -25 * np.sqrt(T * F)
            assert abs((grad * d).sum() - want) <= 5 * (pm.HALF_STEP[dtype] * np.linalg.norm(grad) + small) + own


def single(G, U, dtype):
    """dw_gate, dw_up of one token whose only input is 1, with dh = 1: the kept factors, rounded."""
    F = len(G)
    x = torch.zeros(1, 8, dtype=dtype)
    x[0, 0] = 1
    wg, wu = torch.zeros(F, 8, dtype=dtype), torch.zeros(F, 8, dtype=dtype)
    wg[:, 0], wu[:, 0] = torch.from_numpy(G).to(dtype), torch.from_numpy(U).to(dtype)
    _, g, u = forward(x.cuda(), wg.cuda(), wu.cuda())
    _, dwg, dwu = backward(torch.ones(1, F, dtype=dtype).cuda(), x.cuda(), wg.cuda(), wu.cuda(), g, u)
    return f64(wg)[:, 0], f64(wu)[:, 0], f64(dwg)[:, 0], f64(dwu)[:, 0]


@pytest.mark.parametrize("dtype,lo,hi", [(torch.bfloat16, -80, 58), (torch.float16, -20, 15)])
def test_factors_over_the_exponents(dtype, lo, hi):
    """Either factor anywhere in the range, the other of unit size."""
    rng = np.random.default_rng(17)
    F = 4096
    G, U, dwg, dwu = single(rng.standard_normal(F), rng.choice([-1.0, 1.0], F) * 2.0 ** rng.uniform(lo, hi, F), dtype)
    s = pm.sigmoid(G)
    r, z, e32 = pm.HALF_STEP[dtype], subnormal(dtype), 10 * 2.0 ** -24
    for got, want, e in ((dwg, U * s * (1 + G * (1 - s)), e32 * np.abs(U) * s * (1 + np.abs(G) * (1 + s))),
                         (dwu, G * s, e32 * np.abs(G) * s)):
        off = e + kept(np.abs(want) + e, dtype)
        assert (np.abs(got - want) <= off * (1 + r) + r * np.abs(want) + z).all()


def test_a_factor_out_of_range_leaves_the_other():
    """A factor beyond what is held is infinite or NaN, and the gradient of the other is as ever."""
    for dtype, big in ((torch.bfloat16, 2.0 ** 70), (torch.float16, 65504.0)):
        G = np.full(64, 2.5)                       # dh/dg = 1.09 u: past 65504 in fp16
        G, U, dwg, dwu = single(G, np.full(64, big), dtype)
        assert not np.isfinite(dwg).any()
        want = G * pm.sigmoid(G)
        assert (np.abs(dwu - want) <= 2 * pm.HALF_STEP[dtype] * want).all()

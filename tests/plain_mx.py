"""Plain 64-bit forms of the MXFP4 and gated operators, and the error bounds of their kernels.

Nothing here is shared with the library.  Roundings are counted: a value held in a type is
off by at most eps/2 of it; a sum of n fp32 terms, whatever its order and whether its
additions round or truncate, by at most n * 2^-23 of the sum of magnitudes.
"""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
SUM = 2.0 ** -23


def quantize(x):
    """64-bit rows [..][K] -> (codes 0..15 [..][K], scale bytes [..][K/32])."""
    b = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    _, e = np.frexp(amax)                        # amax = m 2^e, m in [1/2, 1)
    e = np.where(amax > 0, np.maximum(e - 1 - 2, -127), -127)
    v = np.abs(np.ldexp(b, -e[..., None]))
    # nearest of the grid, ties to the even code, magnitudes above 6 held as 6
    d = np.abs(np.minimum(v, 6.0)[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(b))
    return code.reshape(np.shape(x)).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def values(code, scale):
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def held(x):
    """The values that x's MXFP4 codes stand for."""
    return values(*quantize(x))


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def gate(x, wg, wu):
    """(g, u, h, bound of the kernel's fp32 h, bounds of g and u) in 64 bits."""
    g, u = x @ wg.T, x @ wu.T
    k = x.shape[-1]
    eg, eu = k * SUM * (np.abs(x) @ np.abs(wg).T), k * SUM * (np.abs(x) @ np.abs(wu).T)
    s = sigmoid(g)
    h = g * s * u
    # |silu'| <= 1.1; the exponential, the quotient and two products: 8 roundings at most
    eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(g * s) * eu + 8 * 2.0 ** -24 * np.abs(h)
    return g, u, h, eh, eg, eu


def quantize_slack(h, eh):
    """How far the MXFP4 value of a number within eh of h can be from h's own: nothing where both
    round the same way, else the spread of what lies between."""
    lo, hi = h - eh, h + eh
    b = lambda v: v.reshape(*v.shape[:-1], -1, 32)  # noqa: E731
    mags = np.maximum(np.abs(b(lo)), np.abs(b(hi)))
    small = np.where(np.sign(b(lo)) == np.sign(b(hi)), np.minimum(np.abs(b(lo)), np.abs(b(hi))), 0.0)
    tops = []
    for m in (small.max(-1), mags.max(-1)):      # the least and the largest scale of the block
        _, e = np.frexp(m)
        tops.append(np.where(m > 0, e - 3, -127))
    own = held(h)
    slack = np.zeros_like(own)
    for e in tops:
        for v in (lo, hi):
            w = np.ldexp(b(v), -e[..., None])
            step = np.where(np.abs(w) < 2, 0.5, np.where(np.abs(w) < 4, 1.0, 2.0))
            q = np.clip(np.round(w / step) * step, -6, 6)
            q = np.ldexp(q, e[..., None]).reshape(h.shape)
            slack = np.maximum(slack, np.abs(q - own))
    return slack

"""Reference of the block-scaled e4m3 products on the host in float64, and how far a right result may be
from it.  The contract is include/sq_fp8.h's.

Rounding of rows and weights is exact arithmetic (a power of two, then one rounding of the value), so the
codes are those of the library bit for bit wherever its inputs are given.  What is left:
  sums       a tensor-core step adds 32 products to an fp32 sum.  The products of codes and scales are
             exact; the sum is cut to fp32 (at most one unit, 2^-23 of its magnitude), and so are the
             products where they are aligned to it (as much again): 2^-22 of the magnitudes summed so
             far, ceil(L / 32) times, so  L / 32 * 2^-22 * sum|x||W|  (blocks of 128: L rounded up).
  act        sigmoid(v) from e^-|v|, whose error is (2 + 1.16 |v|) units of 2^-23, a sum, a quotient and
             products of one to two units each: (8 + 2.4 |v|) 2^-23 of the value, v = g, or 2 z of the
             gelu, whose own rounding (4 operations on a relative scale) moves sigmoid by at most
             |v| 2^-21 of the value.
  dg, du     three products more, and in act' a sum of s and g w, each with act's error.
A value of dg or du that lies nearer to a rounding border than its error may be rounded to the other side;
what that does to the result is part of the bound (`doubt`).
A bf16 result adds 2^-8 of the value.
"""
import numpy as np

from w8a8ref import bf16, check  # noqa: F401

U23 = 2.0 ** -23
B = 128


def nblocks(n):
    return (n + B - 1) // B


def exponent(top):
    """The least e >= -127 with top <= 448 2^e (top 0: -127)."""
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(np.where(top > 0, top, 1.0) / 448.0))
    e = np.where(448.0 * 2.0 ** (e - 1) >= top, e - 1, e)
    e = np.where(448.0 * 2.0 ** e < top, e + 1, e)
    return np.maximum(np.where(top > 0, e, -127), -127)


def e4m3(t):
    """t (|t| <= 448) rounded to e4m3, to nearest even."""
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -6))) - 3)
    return np.rint(t / step) * step


def blocked(r):
    w = r.shape[1]
    return np.pad(r, ((0, 0), (0, -w % B))).reshape(r.shape[0], -1, B)


def rounded(r, top=None):
    """Rows r [M, L] float64 after the rounding; rows with a NaN or an infinity are NaN.  top: another
    maximum of each block to take the scale from."""
    b = blocked(r)
    fine = np.isfinite(b).all(axis=2, keepdims=True)
    b = np.where(fine, b, 0.0)
    s = 2.0 ** exponent(np.abs(b).max(axis=2, keepdims=True) if top is None else top)
    out = np.where(fine, e4m3(np.clip(b / s, -448, 448)) * s, np.nan)
    return out.reshape(r.shape[0], -1)[:, :r.shape[1]]


def doubtful(r, err):
    """rounded(r) and the most that it can move when r is known to +- err."""
    q = rounded(r)
    fine = np.isfinite(r) & np.isfinite(err)
    top, e = np.abs(blocked(np.where(fine, r, 0.0))), blocked(np.where(fine, err, 0.0))
    most = np.zeros_like(q)
    for t in (np.maximum(top - e, 0).max(axis=2, keepdims=True), (top + e).max(axis=2, keepdims=True)):
        for v in (r - err, r + err):
            most = np.maximum(most, np.abs(rounded(v, t) - q))
    return q, most


def build(W):
    """(codes as values float64 [N, K], scale bytes uint8) of a weight; NaN codes where W is not finite."""
    N, K = W.shape
    W = W.astype(np.float64)
    fine = np.isfinite(W)
    p = np.pad(np.where(fine, np.abs(W), 0.0), ((0, -N % B), (0, -K % B))).reshape(nblocks(N), B, nblocks(K), B)
    e = exponent(p.max(axis=(1, 3)))
    full = np.repeat(np.repeat(e, B, 0), B, 1)[:N, :K]
    return np.where(fine, e4m3(np.where(fine, W, 0.0) * 2.0 ** -full), np.nan), (e + 127).astype(np.uint8)


def dequant(q, s):
    """W float64 from code values [N, K] and scale bytes."""
    N, K = q.shape
    return q * np.repeat(np.repeat(2.0 ** (s.astype(np.float64) - 127), B, 0), B, 1)[:N, :K]


def product(r, W, doubt=None):
    """r W^T in float64 with the bound of an fp32 result."""
    L = nblocks(r.shape[1]) * B
    y = r @ W.T
    bound = L / 32 * 2 * U23 * (np.abs(r) @ np.abs(W).T)
    if doubt is not None:
        bound = bound + doubt @ np.abs(W).T
    return y, bound


def sigmoid(v):
    return np.where(v < 0, np.exp(-np.abs(v)), 1.0) / (1 + np.exp(-np.abs(v)))


C2 = 2 * np.sqrt(2 / np.pi)


def act(g, kind):
    """act(g), act'(g) and their error bounds (absolute)."""
    v = g if kind == "silu" else C2 * (g + 0.044715 * g ** 3)
    dv = np.ones_like(g) if kind == "silu" else C2 * (1 + 3 * 0.044715 * g * g)
    s, w = sigmoid(v), sigmoid(v) * sigmoid(-v)
    eps = (8 + 2.4 * np.abs(v) + (4 * np.abs(v) if kind == "gelu" else 0)) * U23
    return g * s, s + g * w * dv, eps * np.abs(g * s), 2 * eps * (s + np.abs(g * w * dv))


def forward(x, W):
    return product(rounded(x.astype(np.float64)), W)


def backward(dy, W):
    return product(rounded(dy.astype(np.float64)), W.T)


def gated_forward(x, Wg, Wu, kind):
    """((h, bound), (g, bound), (u, bound))"""
    r = rounded(x.astype(np.float64))
    (g, bg), (u, bu) = product(r, Wg), product(r, Wu)
    a, _, ea, _ = act(g, kind)
    ea = ea + 1.13 * bg                                      # |act'| <= 1.13
    h = a * u
    return (h, ea * np.abs(u) + (np.abs(a) + ea) * bu + U23 * np.abs(h)), (g, bg), (u, bu)


def gated_backward(dh, g, u, Wg, Wu, kind):
    dh, g, u = (v.astype(np.float64) for v in (dh, g, u))
    a, slope, ea, es = act(g, kind)
    dg, du = dh * u * slope, dh * a
    qg, mg = doubtful(dg, np.abs(dh * u) * es + 3 * U23 * np.abs(dg))
    qu, mu = doubtful(du, np.abs(dh) * ea + 2 * U23 * np.abs(du))
    (p, bp), (q, bq) = product(qg, Wg.T, mg), product(qu, Wu.T, mu)
    return p + q, bp + bq + U23 * np.abs(p + q)


def layer(rng, N, K, E=None):
    """Random codes (values as fp32) and scale bytes."""
    lead = () if E is None else (E,)
    q = e4m3(np.clip(rng.standard_normal(lead + (N, K)) * 90, -448, 448)).astype(np.float32)
    return q, (rng.integers(-2, 3, lead + (nblocks(N), nblocks(K))) + 113).astype(np.uint8)

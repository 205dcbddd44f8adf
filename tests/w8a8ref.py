"""Reference of the 8-bit integer products on the host, and how far a right result may be from it.

codes(): the row quantisation operation by operation in numpy float32, one rounding each, as the
contract in include/sq_w8a8.h states it.  forward() and backward(): the product from those codes in
float64, with a bound on the library's fp32 arithmetic, element by element.  u = 2^-24 is half a
step of fp32, 2^-8 half a step of bf16 (relative to the value):
  main term   RN(float(acc) RN(s_x s_w)): three roundings, 3 u |main| (4 u with the second-order
              terms); backward RN(float(acc) s_g): two, then eight butterfly stages of one rounding
              per value.  Each stage's rounding is at most u times the sum of magnitudes that
              reaches the element, so the rotation adds 8 u H|main| (H|.|: every sign positive,
              1 / 16 of the sum of magnitudes); 12 u H|main| covers both.
  low rank    t: fp32 sum of K products in some order, at most K u sum|x D|; t . U: 16 more
              products.  (K + 20) u |x| |D| |U| covers both (n u / (1 - n u) for n <= 16384 + 20).
  sum         one rounding of the result, u |y|.
A bf16 result adds its own rounding (2^-8 of the value); backward it takes u as two bf16 terms:
each rounding leaves at most 2^-8 of what is left, so 2^-16 |u| . |D|.
"""
import numpy as np

U24 = 2.0 ** -24
RANK = 16


def bf16(a):
    """fp32 array rounded to bf16 (to nearest even), as fp32."""
    b = np.ascontiguousarray(a, np.float32).view(np.uint32)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def rotate32(v):
    """H256 on each 256-block of the rows of v, radix-2 butterflies in float32."""
    v = np.asarray(v, np.float32)
    k = np.arange(v.shape[1])
    for h in (1, 2, 4, 8, 16, 32, 64, 128):
        other = v[:, k ^ h]
        v = np.where((k & h) == 0, v + other, other - v)
    return v * np.float32(0.0625)


def hadamard():
    k = np.arange(256)
    ones = np.array([bin(i).count("1") for i in range(256)])
    return np.where(ones[k[:, None] & k[None, :]] % 2 == 0, 1.0, -1.0) / 16.0


def blocks(v, H):
    return (v.reshape(v.shape[0], -1, 256) @ H).reshape(v.shape)


def codes(r):
    """(codes float64 [M, K], scales float32 [M]) of the rows r (float32)."""
    r = np.asarray(r, np.float32)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        a = np.abs(r).max(axis=1)
        s = a / np.float32(127)
        s = np.where(np.isfinite(r).all(axis=1), np.where(s < np.float32(2.0) ** -120, np.float32(0), s), np.float32(np.nan))
        inv = np.where(s > 0, np.float32(1) / np.where(s > 0, s, np.float32(1)), np.float32(0))
        q = np.clip(np.rint(r * inv[:, None]), -127, 127)
    return np.where(np.isfinite(s)[:, None], np.nan_to_num(q), 0).astype(np.float64), s.astype(np.float32)


def forward(x, Q, sw, up=None, down=None, bf16_out=False):
    """x [M, K] (bf16 values as fp32), Q [N, K] int8, sw [N] fp32 -> (y float64, bound on an fp32 y).
    bf16_out is backward's and changes nothing here."""
    q, s = codes(rotate32(x))
    main = (q @ Q.astype(np.float64).T) * s.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    y, bound = main, 4 * U24 * np.abs(main)
    if up is not None:
        x64, U, D = x.astype(np.float64), up.astype(np.float64), down.astype(np.float64)
        y = main + (x64 @ D) @ U.T
        bound = bound + (x.shape[1] + 20) * U24 * ((np.abs(x64) @ np.abs(D)) @ np.abs(U).T)
    return y, bound + U24 * np.abs(y)


def backward(dy, Q, sw, up=None, down=None, bf16_out=False):
    """dy [M, N] (bf16 values as fp32) -> (dx [M, K] float64, bound on an fp32 dx)."""
    q, s = codes(dy.astype(np.float32) * sw[None, :].astype(np.float32))
    main = (q @ Q.astype(np.float64)) * s.astype(np.float64)[:, None]
    H = hadamard()
    dx, bound = blocks(main, H), 12 * U24 * blocks(np.abs(main), np.abs(H))
    if up is not None:
        d64, U, D = dy.astype(np.float64), up.astype(np.float64), down.astype(np.float64)
        dx = dx + (d64 @ U) @ D.T
        bound = bound + (dy.shape[1] + 20) * U24 * ((np.abs(d64) @ np.abs(U)) @ np.abs(D).T)
        if bf16_out:
            bound = bound + 2.0 ** -16 * (np.abs(d64 @ U) @ np.abs(D).T)
    return dx, bound + U24 * np.abs(dx)


def check(got, ref, bound, is_bf16):
    """got (float array) within the bound of ref, bf16 outputs one rounding more; NaN rows the same."""
    got = np.asarray(got, np.float64)
    nan = np.isnan(ref)
    assert np.array_equal(nan, np.isnan(got)), "NaN in other places"
    if is_bf16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    off = np.abs(got - ref) - bound
    off[nan] = -1.0
    worst = np.unravel_index(np.argmax(off), off.shape)
    assert off[worst] <= 0, (f"{(off > 0).sum()} of {off.size} out of bound, worst at {worst}: got {got[worst]}, "
                             f"expected {ref[worst]} +- {bound[worst]}")


def layer(rng, N, K, lora=True, E=None):
    """Random int8 layer(s): Q, sw, up, down as numpy (up, down bf16 values in fp32, or None)."""
    lead = () if E is None else (E,)
    Q = np.clip(np.rint(rng.standard_normal(lead + (N, K)) * 40), -127, 127).astype(np.int8)
    sw = ((rng.random(lead + (N,)) + 0.5) * 1e-3).astype(np.float32)
    if not lora:
        return Q, sw, None, None
    return (Q, sw, bf16(rng.standard_normal(lead + (N, RANK)) * 0.2),
            bf16(rng.standard_normal(lead + (K, RANK)) * (0.6 / np.sqrt(K))))

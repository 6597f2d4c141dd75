"""The 8-bit integer cast, product and MLP in 64 bits, with bounds on what an
fp32 evaluation may be off, for the tests."""
import numpy as np

U = 2.0 ** -24                   # half a step of fp32, relative to the value
LEAST = 2.0 ** -100


def top_of(x):
    return np.maximum(np.abs(x).max(1), LEAST)


def cast(x, weight=None):
    """Codes and scales of x (values of fp32 or fewer bits, as float64). 127 x has
    31 bits, so it is exact, and the quotient is either a half or further from one
    than its rounding to 53 bits. The scales' roundings are those of fp32."""
    top = top_of(x)
    q = np.rint(127.0 * x / top[:, None]).astype(np.int64)
    s = top.astype(np.float32) / np.float32(127.0)
    return q, s if weight is None else s * weight.astype(np.float32)


def product(a, a_s, b, b_s):
    """C and its bound: the sum is exact, then rounded to fp32 and multiplied twice."""
    c = (a.astype(np.float64) @ b.astype(np.float64).T) * a_s.astype(np.float64)[:, None] * b_s.astype(np.float64)
    return c, 3.01 * U * np.abs(c)


def mlp(x, probs, w1, w1_s, w2, w2_s):
    """One expert's rows: y and its bound (before the rounding to bf16).

    H's bound is the product's. A = silu(g) u: a relative error d of g changes
    silu(g) by at most (1 + |g|) d relative, and exp, quotient and products add a
    few half steps more, those of exp growing with its argument. A code may be one
    off only where the quotient is as near to a half as 127 times the relative
    errors of the value and of the row's top; then the value is off by a step."""
    q, s = cast(x)
    h, _ = product(q, s, w1, w1_s)
    F = w1.shape[0] // 2
    g, u = h[:, :F], h[:, F:]
    a = g / (1 + np.exp(-np.minimum(np.maximum(g, -700), 700))) * u
    rel = (3.01 * (2 + np.abs(g)) + 8 + 4 * np.abs(g)) * U
    top = top_of(a)
    rel_top = np.where(np.abs(a) * (1 + rel) >= top[:, None] * (1 - rel), rel, 0).max(1)[:, None]
    t = 127 * a / top[:, None]
    code = np.rint(t)
    near = np.abs(np.abs(t - np.floor(t)) - 0.5) <= np.abs(t) * (rel + rel_top + 4 * U)
    step = top / 127 * (1 if probs is None else probs)
    # the sum of integers first, where it is exact: a sum of 0 has to be 0
    y = (code @ w2.astype(np.float64).T) * step[:, None] * w2_s.astype(np.float64)
    size = np.abs(w2.astype(np.float64) * w2_s.astype(np.float64)[:, None]).T
    # where no code flips y is the same integer sum times a scale that is off by rel_top
    return y, (near * step[:, None]) @ size * (1 + 1e-5) + np.abs(y) * (rel_top + 6 * U)

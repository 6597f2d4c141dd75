"""Plain 64-bit forms of the few-row products, the few-token MoE MLP and the
router, with elementwise error bounds of the kernels' arithmetic.

Bounds. Every weight is exact in bf16 and every product of two bf16 numbers is
exact in fp32, so only the sums round. One matrix instruction adds 32 products
to its fp32 accumulator; its result is off by at most 2^-22 of the sum of the
magnitudes it adds (two roundings to nearest, or one truncation, of 2^-23 each
at that magnitude). Along k there are k / 32 instructions, in up to 16 waves
whose results are then added: (k / 32 + 17) * 2^-22 * sum |x| |w| in all. A
result rounded to bf16 is off by half a step more, 2^-8 of its value
(torch.finfo(bfloat16).eps / 2)."""
import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


def e2m1_values(q):
    """Packed codes uint8 [..., k/2] -> float64 [..., k]."""
    q = np.asarray(q)
    nib = np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)
    return np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]


def e4m3_values(c):
    c = np.asarray(c).astype(np.int64)
    man, ex = c & 7, (c >> 3) & 15
    v = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def mxfp4(q, s):
    return e2m1_values(q) * np.repeat(2.0 ** (np.asarray(s).astype(np.float64) - 127), 32, axis=-1)


def mxfp8(q, s):
    return e4m3_values(q) * np.repeat(2.0 ** (np.asarray(s).astype(np.float64) - 127), 32, axis=-1)


def nvfp4(q, s, amax):
    """amax: the tensor's, float."""
    scale = 1.0 if amax == 0 else min(float(np.float32(2688.0) / np.float32(amax)), 2.0 ** 64)
    return e2m1_values(q) * np.repeat(e4m3_values(s), 16, axis=-1) / scale


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def sum_bound(k, mag):
    return (k / 32 + 17) * 2.0 ** -22 * mag


def products(x, w, bf16_out):
    """x [m, k] . w [n, k]^T -> (values, bound)."""
    y = x @ w.T
    b = sum_bound(x.shape[1], np.abs(x) @ np.abs(w).T)
    return y, b + BF16_HALF * (np.abs(y) + b) * bf16_out


def moe(x, idx, wt, w1, w2):
    """x [T, H], idx [T, k] (out of range: dropped), wt [T, k], w1 [E, 2F, H],
    w2 [E, H, F] -> (y, bound). The first product is off by its sums' bound;
    silu has a slope of at most 1.1 and its fp32 steps (exp, sum, quotient,
    two products) at most 2^-20 of the value; A as two bf16 numbers keeps
    2^-16 of its value (half a step of each)."""
    T, H = x.shape
    E, F2, _ = w1.shape
    F = F2 // 2
    y, b = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        terms = np.zeros(H)
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if e < 0 or e >= E:
                continue
            h = w1[e] @ x[t]
            hb = sum_bound(H, np.abs(w1[e]) @ np.abs(x[t]))
            g, u, gb, ub = h[:F], h[F:], hb[:F], hb[F:]
            silu = g / (1 + np.exp(-g))
            a = wt[t, j] * silu * u
            ab = np.abs(wt[t, j]) * (1.1 * gb * (np.abs(u) + ub) + np.abs(silu) * ub) + (2.0 ** -20 + 2.0 ** -16) * np.abs(a)
            y[t] += w2[e] @ a
            b[t] += np.abs(w2[e]) @ ab
            terms += np.abs(w2[e]) @ (np.abs(a) + ab)
        b[t] += sum_bound(F * idx.shape[1], terms)
    return y, b + BF16_HALF * (np.abs(y) + b)


def route(z, bias, k, renorm):
    """z float32 [T, E] (the logits' values), bias float32 [E] or None ->
    (idx, w, lse, relative bound of w, absolute bound of lse). Keys are formed in fp32, as defined."""
    z = np.asarray(z, dtype=np.float32)
    T, E = z.shape
    with np.errstate(invalid="ignore"):
        key = z if bias is None else (z + np.asarray(bias, dtype=np.float32)[None]).astype(np.float32)
        open_ = key > -np.inf
    key = np.where(open_, key, -np.inf)
    order = np.argsort(-key.astype(np.float64), axis=1, kind="stable")[:, :k]
    taken = np.take_along_axis(open_, order, 1)
    idx = np.where(taken, order, -1).astype(np.int32)
    zd = np.where(open_, z, -np.inf).astype(np.float64)
    top = zd.max(axis=1, keepdims=True)
    ref = np.where(np.isfinite(top), top, 0.0)
    total = np.exp(zd - ref).sum(1)
    with np.errstate(divide="ignore"):
        lse = np.log(total) + np.where(total > 0, ref[:, 0], 0.0)
    zk = np.where(taken, np.take_along_axis(zd, order, 1), -np.inf)
    if renorm:
        r = zk.max(axis=1, keepdims=True)
        ek = np.exp(zk - np.where(np.isfinite(r), r, 0.0))
        s = ek.sum(1, keepdims=True)
        w = np.where(s > 0, ek / np.where(s > 0, s, 1.0), 0.0)
    else:
        w = np.where(taken, np.exp(zk - np.where(np.isfinite(lse), lse, 0.0)[:, None]), 0.0)
    # exp of a difference d of fp32 numbers: |d| 2^-24 from the rounding of d, 2 ulp of the
    # function; the sum of E such terms: E 2^-24 more; a quotient: 2^-24
    spread = np.where(np.isfinite(zd), np.abs(zd - ref), 0.0).max(axis=1, keepdims=True)
    rel = (2 * spread + E + 16) * 2.0 ** -23
    lse_b = rel[:, 0] + np.where(np.isfinite(lse), np.abs(lse), 0.0) * 2.0 ** -22
    return idx, w, lse, rel, lse_b


def route_bwd(z, bias, idx, w, lse, dw, renorm):
    """All float64 (idx int) with the forward's own w and lse -> (dz, bound of its fp32 steps)."""
    z = np.asarray(z, dtype=np.float64)
    T, E = z.shape
    ok = (idx >= 0) & (idx < E)
    wd = np.where(ok, w * np.where(ok, dw, 0.0), 0.0)
    dot, mag = wd.sum(1, keepdims=True), np.abs(wd).sum(1, keepdims=True)
    k = idx.shape[1]
    dz, b = np.zeros((T, E)), np.zeros((T, E))
    if not renorm:
        with np.errstate(invalid="ignore"):
            open_ = (z if bias is None else z + bias[None]) > -np.inf
        d = np.where(open_, z - np.where(np.isfinite(lse), lse, 0.0)[:, None], 0.0)
        p = np.where(open_, np.exp(d), 0.0)
        dz -= p * dot
        b += p * mag * (k + 8 + 2 * np.abs(d)) * 2.0 ** -23
    for t in range(T):
        for j in range(k):
            if ok[t, j]:
                dz[t, idx[t, j]] += wd[t, j] - (w[t, j] * dot[t, 0] if renorm else 0.0)
                b[t, idx[t, j]] += (np.abs(wd[t, j]) + w[t, j] * mag[t, 0]) * (k + 8) * 2.0 ** -23
    return dz, b

"""The balance loss, its sums and its gradient in 64 bits, with bounds on what an
fp32 evaluation may be off, for the tests."""
import numpy as np

U = 2.0 ** -24                   # half a step of fp32, relative to the value


def spans(segments, T):
    if segments is None:
        return [(0, T)]
    o = np.clip(np.asarray(segments, dtype=np.int64), 0, T)
    return [(b, max(b, e)) for b, e in zip(o[:-1], o[1:])]


def probs(z, bias):
    """(p [T, E], relative error bound [T, E]) of a softmax over the open experts:
    z - max is rounded once (an error of |z - max| U in the exponent), exp is good
    to two half steps, the sum has at most 12 additions in a chain, and the
    reciprocal and the product round once each. Zeros where nothing is open."""
    key = z if bias is None else z + bias
    open_ = key > -np.inf
    zz = np.where(open_, z, -np.inf)
    top = zz.max(1, keepdims=True)
    far = np.where(open_, np.where(open_, top, 0) - np.where(open_, z, 0), 0.0)
    e = np.where(open_, np.exp(-far), 0.0)
    total = e.sum(1, keepdims=True)
    p = e / np.where(total > 0, total, 1)
    own = far * U + 2 * U
    return p, own + (p * own).sum(1, keepdims=True) + 14 * U


def balance(z, bias, idx, segments, E):
    """loss, counts, mean_prob, and the bounds of loss and mean_prob."""
    T, k = idx.shape
    p, rel = probs(z, bias)
    loss, counts, mean, bl, bm = [], [], [], [], []
    for b, e in spans(segments, T):
        n = max(1, e - b)
        ids = idx[b:e].reshape(-1)
        c = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        m, mb = p[b:e].sum(0) / n, (p[b:e] * rel[b:e]).sum(0) / n
        mb = mb + U * m                                      # the sums are 64 bits; rounded once
        counts.append(c)
        mean.append(m)
        bm.append(mb)
        loss.append(E / (k * n) * (c * m).sum())
        bl.append(E / (k * n) * (c * mb).sum() + U * loss[-1])
    return np.array(loss), np.array(counts), np.array(mean), np.array(bl), np.array(bm)


def balance_bwd(z, bias, counts, k, dloss, dmean, segments, add):
    """dlogits and its bound (before a rounding to the logits' type). A is rounded
    to fp32 after its mean over the experts is taken off, which the gradient does
    not see; p (A - dot) multiplies three rounded numbers."""
    T, E = z.shape
    p, rel = probs(z, bias)
    dz, bound = np.zeros((T, E)), np.zeros((T, E))
    for s, (b, e) in enumerate(spans(segments, T)):
        if e == b:
            continue
        n = e - b
        A = np.zeros(E)
        if dloss is not None:
            A = A + dloss[s] * E / (k * n) * counts[s]
        if dmean is not None:
            A = A + dmean[s]
        A = (A - A.mean()) / n
        # the mean taken off is an fp32 sum, so it may be off, by at most 12 U of the largest
        size = np.abs(A) + 12 * U * np.abs(A).max()
        pp, rr = p[b:e], rel[b:e]
        dot = (pp * A).sum(1, keepdims=True)
        off = (pp * size * (rr + 12 * U)).sum(1, keepdims=True)
        dz[b:e] = pp * (A - dot)
        bound[b:e] = pp * ((rr + 3 * U) * (np.abs(A - dot) + off) + U * size + off)
    if add is not None:
        dz = dz + add
        bound = bound + U * (np.abs(dz) + bound)
    return dz, bound

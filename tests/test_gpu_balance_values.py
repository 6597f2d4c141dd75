"""Values at the border of what the balance loss (mx_moe_balance,
mx_moe_balance_bwd) takes: what is not finite shows, and only where it belongs;
gradients of the means that are far apart, or that share a large part; the
exponential over its range."""
import numpy as np
import pytest
import torch

from tests import balance_ref as ref
from tests import decode_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [1, 5, 8, 60, 128])
@pytest.mark.parametrize("T", [40, 700])                  # one part a sequence, and several
def test_infinite_logits_show(gpu_lib, T, E, dtype):
    """A logit of +inf makes its token's softmax NaN (inf - inf), so the loss and
    the means of its sequence and the token's gradient are, and no others."""
    gen = torch.Generator().manual_seed(T + E)
    k = min(2, E)
    z = torch.randn((T, E), generator=gen).to(dtype).cuda()
    idx = gpu_lib.mx_moe_route(z, k)[0]
    seg = torch.tensor([0, T // 4, T // 2, T - 3], dtype=torch.int32, device="cuda")
    dl, dm = torch.randn(3, generator=gen).cuda(), torch.randn((3, E), generator=gen).cuda()
    add = torch.randn((T, E), generator=gen).to(dtype).cuda()

    def run(logits, bias=None):
        loss, counts, mean = gpu_lib.mx_moe_balance(logits, idx, bias=bias, segments=seg)
        dz = gpu_lib.mx_moe_balance_bwd(logits, counts, k, dloss=dl, dmean_prob=dm, bias=bias, segments=seg, add=add)
        return loss, counts, mean, dz

    want = run(z)
    bad = z.clone()
    rows = [T // 4 + 1, T // 2 - 1]                        # both of the second sequence
    bad[rows[0], E // 2] = float("inf")
    bad[rows[1]] = float("inf")
    bad[T - 1, 0] = float("inf")                           # behind the last sequence: takes no part
    loss, counts, mean, dz = run(bad)
    assert torch.isnan(loss[1]) and torch.isnan(mean[1]).all() and torch.isnan(dz[rows]).all()
    assert torch.equal(counts, want[1])
    assert torch.equal(loss[[0, 2]], want[0][[0, 2]]) and torch.equal(mean[[0, 2]], want[2][[0, 2]])
    rest = np.setdiff1d(np.arange(T), rows)
    assert torch.equal(dz[rest], want[3][rest])
    # shut by its key (inf - inf is NaN): as if it were not there
    if E > 1:
        b = torch.zeros(E, device="cuda")
        b[0] = float("-inf")
        shut = z.clone()
        shut[:, 0] = float("inf")
        assert all(torch.equal(x, y) for x, y in zip(run(shut, b), run(z, b)))


def _gradient(z, dm, segments):
    """dlogits of the means' gradients dm in 64 bits, and its bound, with the p and
    their relative bounds r of balance_ref. a = A - c, rounded once, with c the point
    between the least and the largest A that is nearest to 0: the softmax does not
    see it, equal A become 0, and |a| <= |A|. With b = a - dot the sum over p b has
    p's errors, b's and a product's rounding and at most 9 additions, so whatever
    dot's error was, what is left of it is relative to sum p |b|; a difference and
    a product round after that."""
    u = ref.U
    p, r = ref.probs(z, None)
    dz, bound = np.zeros_like(z), np.zeros_like(z)
    for s, (b, e) in enumerate(ref.spans(segments, len(z))):
        A = dm[s] / max(1, e - b)
        a = (A - np.clip(0, A.min(), A.max()))[None]
        pp, rr = p[b:e], r[b:e]
        diff = a - (pp * a).sum(1, keepdims=True)
        off = (pp * (u * np.abs(a) + (rr + 11 * u) * np.abs(diff))).sum(1, keepdims=True)
        dz[b:e] = pp * diff
        bound[b:e] = 1.01 * pp * ((rr + 3 * u) * np.abs(diff) + u * np.abs(a) + off)
    return dz, bound


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [5, 8, 60, 128])
@pytest.mark.parametrize("kind", ["rare", "rare and positive", "rare with offset", "offset", "negative offset"])
def test_gradients_of_means_far_apart(gpu_lib, E, kind, dtype):
    """The gradient of sum log mean_prob, where one expert's mean is next to
    nothing and its gradient that much larger than the others'; and gradients that
    share a part a thousand times what differs."""
    T, o = 300, [0, 170, 300]
    gen = torch.Generator().manual_seed(E)
    z = torch.randn((T, E), generator=gen)
    if "rare" in kind:
        z[:170, 3] -= 22.0
    z = z.to(dtype).cuda()
    seg = torch.tensor(o, dtype=torch.int32, device="cuda")
    mean = gpu_lib.mx_moe_balance(z, gpu_lib.mx_moe_route(z, 2)[0], segments=seg)[2]
    if "rare" in kind:
        assert mean[0, 3] < 1e-8
        dm = 1 / (E * mean) if "positive" in kind else -1 / (E * mean)
        if "offset" in kind:
            dm = dm + 1000.0
    else:
        dm = torch.randn((2, E), generator=gen).cuda() + (1000.0 if kind == "offset" else -1000.0)
    dz = gpu_lib.mx_moe_balance_bwd(z, None, 2, dmean_prob=dm, segments=seg)
    want, bound = _gradient(decode_ref.f64(z), decode_ref.f64(dm), o)
    if dtype == torch.bfloat16:
        bound = bound + decode_ref.BF16_HALF * (np.abs(want) + bound)
    assert np.all(np.abs(decode_ref.f64(dz) - want) <= bound + 1e-37)


def test_probabilities_over_the_range(gpu_lib):
    """Tokens of their own sequences with logits 0 and -x: the mean is p = e / (1 +
    e) itself. e = exp(-x) is good to three half steps (the difference to the
    maximum is exact), 1 + e rounds once, the reciprocal is good to two and the
    product to one: 7 for p, and e's again by its share of the sum. Results below
    2^-126 may be 0."""
    S = 60000
    x = torch.linspace(0, 120, S, dtype=torch.float32)
    z = torch.stack([torch.zeros(S), -x], 1).cuda()
    seg = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    mean = decode_ref.f64(gpu_lib.mx_moe_balance(z, gpu_lib.mx_moe_route(z, 1)[0], segments=seg)[2])
    e = np.exp(-x.double().numpy())
    p = e / (1 + e)
    assert np.all(np.abs(mean[:, 1] - p) <= 1.001 * (7 + 3 * p) * ref.U * p + 2.0 ** -126)
    assert np.all(np.abs(mean[:, 0] - (1 - p)) <= 1.001 * (4 + 3 * p) * ref.U)

"""The balance loss (mx_moe_balance, mx_moe_balance_bwd, MoEBalance) against the
64-bit form: counts exactly, losses, means and gradients within derived bounds;
ragged and empty sequences, padding, shut experts, streams, graphs."""
import numpy as np
import pytest
import torch

from tests import balance_ref as ref
from tests import decode_ref
from tests.gpu_util import canaries_intact, guarded

pytestmark = pytest.mark.gpu

f64 = decode_ref.f64
SHAPES = [(1, 1, 1), (1, 8, 2), (3, 4, 4), (7, 5, 2), (64, 16, 16), (65, 17, 3), (300, 60, 6), (129, 64, 16), (257, 65, 5),
          (1000, 128, 8), (31, 127, 16), (4099, 8, 2), (16383, 128, 8)]


def _inputs(gpu_lib, T, E, k, dtype, seed, masked=True):
    gen = torch.Generator().manual_seed(seed)
    z = (2 * torch.randn((T, E), generator=gen)).to(dtype)
    if masked:
        z[torch.rand((T, E), generator=gen) < 0.1] = float("-inf")
        if T > 3:
            z[1] = float("-inf")                       # nothing open
            z[2, 1:] = float("-inf")                   # one open
            z[3, 0] = float("nan")                     # shut too
    z, bias = z.cuda(), (0.3 * torch.randn(E, generator=gen)).cuda()
    return z, bias, gpu_lib.mx_moe_route(z, k, bias=bias)[0]


def _segments(T, kind):
    if kind == "all":
        return None
    if kind == "ragged":
        o = sorted({0, T // 3, T // 3 + 1, T // 2, T - T // 7})
        return [o[0], o[0]] + o[1:] + [o[-1]]          # empty ones first and last, padding behind
    return sorted(np.random.default_rng(T).integers(0, T + 1, size=70).tolist())


def _dev(o):
    return None if o is None else torch.tensor(o, dtype=torch.int32, device="cuda")


def _np(z):
    a = f64(z)
    return np.where(np.isnan(a), -np.inf, a)           # a NaN shuts its expert


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_losses_counts_and_gradients(gpu_lib, T, E, k, dtype):
    z, bias, idx = _inputs(gpu_lib, T, E, k, dtype, T + E)
    rng = np.random.default_rng(E)
    for kind in ("all", "ragged", "many"):
        o = _segments(T, kind)
        seg, S = _dev(o), 1 if o is None else len(o) - 1
        b = bias if kind != "ragged" else None
        loss, counts, mean = gpu_lib.mx_moe_balance(z, idx, bias=b, segments=seg)
        bn = None if b is None else b.double().cpu().numpy()
        rl, rc, rm, bl, bm = ref.balance(_np(z), bn, idx.cpu().numpy(), o, E)
        assert counts.dtype == torch.int64 and np.array_equal(counts.cpu().numpy(), rc)
        assert np.all(np.abs(f64(mean) - rm) <= bm) and np.all(np.abs(f64(loss) - rl) <= bl)
        dloss = torch.from_numpy(rng.standard_normal(S).astype(np.float32)).cuda()
        dmean = torch.from_numpy(rng.standard_normal((S, E)).astype(np.float32)).cuda()
        add = torch.randn((T, E), device="cuda").to(dtype) * 1e-3
        for dl, dm, base in ((dloss, None, None), (None, dmean, add), (dloss, dmean, add)):
            dz = gpu_lib.mx_moe_balance_bwd(z, counts if dl is not None else None, k, dloss=dl, dmean_prob=dm, bias=b,
                                            segments=seg, add=base)
            want, bound = ref.balance_bwd(_np(z), bn, rc, k, None if dl is None else f64(dl),
                                          None if dm is None else f64(dm), o, None if base is None else f64(base))
            if dtype == torch.bfloat16:
                bound = bound + decode_ref.BF16_HALF * (np.abs(want) + bound)
            assert dz.dtype == dtype and np.all(np.abs(f64(dz) - want) <= bound + 1e-37)
        # in place: the same bits
        same = add.clone()
        gpu_lib.mx_moe_balance_bwd(z, counts, k, dloss=dloss, dmean_prob=dmean, bias=b, segments=seg, add=same, out=same)
        assert torch.equal(same, dz)


def test_gradient_against_differences(gpu_lib):
    """Central differences of the 64-bit loss and means in every logit: h^2 times a
    third derivative of a softmax (at most 1) times the weights, plus 2^-52 / h."""
    T, E, k, h = 9, 6, 2, 1e-4
    z, _, idx = _inputs(gpu_lib, T, E, k, torch.float32, 5, masked=False)
    o = [0, 4, 4, 8]
    rng = np.random.default_rng(2)
    dl, dm = rng.standard_normal(3).astype(np.float32), rng.standard_normal((3, E)).astype(np.float32)
    _, counts, _ = gpu_lib.mx_moe_balance(z, idx, segments=_dev(o))
    got = f64(gpu_lib.mx_moe_balance_bwd(z, counts, k, dloss=torch.from_numpy(dl).cuda(),
                                         dmean_prob=torch.from_numpy(dm).cuda(), segments=_dev(o)))
    zn, ids = f64(z), idx.cpu().numpy()

    def value(a):
        loss, _, mean, _, _ = ref.balance(a, None, ids, o, E)
        return (loss * dl).sum() + (mean * dm).sum()

    size = np.abs(dl).sum() * E + np.abs(dm).sum()
    for t in range(T):
        for e in range(E):
            up, down = zn.copy(), zn.copy()
            up[t, e] += h
            down[t, e] -= h
            num = (value(up) - value(down)) / (2 * h)
            assert abs(got[t, e] - num) <= size * (h * h + 2.0 ** -50 / h + 64 * 2.0 ** -24)
    assert np.all(got[8] == 0)                              # behind the last sequence


def test_autograd(gpu_lib):
    """MoEBalance against autograd through the definition in 64 bits."""
    T, E, k = 200, 16, 3
    z, bias, idx = _inputs(gpu_lib, T, E, k, torch.float32, 11, masked=False)
    o = [3, 90, 190]
    zz = z.clone().requires_grad_()
    loss, counts, mean = gpu_lib.MoEBalance.apply(zz, idx, bias, _dev(o))
    w = torch.randn((2, E), device="cuda")
    (loss.sum() * 0.3 + (mean * w).sum()).backward()
    z64 = z.double().cpu().requires_grad_()
    p = torch.softmax(z64, 1)
    total = 0.0
    for s, (b, e) in enumerate(zip(o[:-1], o[1:])):
        c = torch.bincount(idx[b:e].reshape(-1).long().cpu(), minlength=E).double()
        assert torch.equal(c.long(), counts[s].cpu())
        m = p[b:e].mean(0)
        total = total + 0.3 * E / (k * (e - b)) * (c * m).sum() + (m * w[s].double().cpu()).sum()
    total.backward()
    want, bound = ref.balance_bwd(f64(z), f64(bias), counts.cpu().numpy(), k, np.full(2, np.float32(0.3)), f64(w), o, None)
    assert np.abs(want - z64.grad.numpy()).max() <= 1e-8 + 2e-8 * np.abs(want).max()       # 0.3 in 32 bits
    assert np.all(np.abs(f64(zz.grad) - want) <= bound)
    # one of the two outputs alone, and neither
    for pick in (0, 2):
        zz = z.clone().requires_grad_()
        gpu_lib.MoEBalance.apply(zz, idx, None, None)[pick].sum().backward()
        assert torch.isfinite(zz.grad).all()
    assert not gpu_lib.MoEBalance.apply(z, idx)[0].requires_grad


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_far_logits(gpu_lib, dtype):
    """Masks of the type's lowest value are open experts of probability 0; rows of
    nothing but them are even; logits far apart."""
    z = torch.randn((40, 20), device="cuda").to(dtype)
    z[3, 5:] = torch.finfo(dtype).min
    z[4] = torch.finfo(dtype).min
    z[5, ::2], z[5, 1::2] = torch.finfo(dtype).min, torch.finfo(dtype).max
    z[6] = (torch.arange(20, device="cuda") * -9.7).to(dtype)
    z[7] = z[6] + 1e4
    idx = gpu_lib.mx_moe_route(z, 3)[0]
    loss, counts, mean = gpu_lib.mx_moe_balance(z, idx)
    zn = f64(z)
    rl, rc, rm, bl, bm = ref.balance(zn, None, idx.cpu().numpy(), None, 20)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.all(np.abs(f64(mean) - rm) <= bm) and np.all(np.abs(f64(loss) - rl) <= bl)
    w = torch.randn((1, 20), device="cuda")
    dz = gpu_lib.mx_moe_balance_bwd(z, counts, 3, dloss=torch.ones(1, device="cuda"), dmean_prob=w)
    want, bound = ref.balance_bwd(zn, None, rc, 3, np.ones(1), f64(w), None, None)
    if dtype == torch.bfloat16:
        bound = bound + decode_ref.BF16_HALF * (np.abs(want) + bound)
    assert np.all(np.abs(f64(dz) - want) <= bound + 1e-37)


def test_choices_outside_and_repeated(gpu_lib):
    z = torch.randn((70, 12), device="cuda")
    idx = torch.randint(0, 12, (70, 4), device="cuda", dtype=torch.int32)
    idx[::3, 1], idx[::5, 2], idx[::7] = -1, 12, 5         # outside, and one expert four times
    _, counts, _ = gpu_lib.mx_moe_balance(z, idx)
    flat = idx.reshape(-1).long()
    assert torch.equal(counts[0], torch.bincount(flat[(flat >= 0) & (flat < 12)], minlength=12))


def test_offsets_outside_are_cut(gpu_lib):
    z, _, idx = _inputs(gpu_lib, 300, 8, 2, torch.float32, 3)
    for o in ([-5, 100, 999], [400, 500], [200, 100, 50], [-(2 ** 31), 2 ** 31 - 1]):
        loss, counts, mean = gpu_lib.mx_moe_balance(z, idx, segments=_dev(o))
        rl, rc, rm, bl, bm = ref.balance(_np(z), None, idx.cpu().numpy(), o, 8)
        assert np.array_equal(counts.cpu().numpy(), rc) and np.all(np.abs(f64(mean) - rm) <= bm)
        dz = gpu_lib.mx_moe_balance_bwd(z, counts, 2, dloss=torch.ones(len(o) - 1, device="cuda"), segments=_dev(o))
        assert torch.isfinite(dz).all()
        inside = np.zeros(300, dtype=bool)
        for b, e in ref.spans(o, 300):
            inside[b:e] = True
        if sorted(o) == o:
            assert np.all(f64(dz)[~inside] == 0)


def test_no_tokens_guards_and_a_side_stream(gpu_lib):
    z, bias, idx = _inputs(gpu_lib, 2000, 60, 6, torch.bfloat16, 3)
    seg = _dev([0, 700, 700, 1900])
    want = gpu_lib.mx_moe_balance(z, idx, bias=bias, segments=seg)
    dl = torch.ones(3, device="cuda")
    wz = gpu_lib.mx_moe_balance_bwd(z, want[1], 6, dloss=dl, bias=bias, segments=seg)
    L, p = gpu_lib.load(), gpu_lib._ptr
    nbytes = gpu_lib.moe_balance_workspace_bytes(2000, 60, 3)
    assert nbytes > 0
    bufs = [guarded(s, d) for s, d in (((3,), torch.float32), ((3, 60), torch.int64), ((3, 60), torch.float32),
                                       ((2000, 60), torch.bfloat16), ((nbytes,), torch.uint8))]
    (_, loss), (_, counts), (_, mean), (_, dz), (_, ws) = bufs
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st = gpu_lib._stream()
        gpu_lib._check(L.mx_moe_balance(p(z), 0, p(bias), p(idx), p(seg), 3, 2000, 60, 6, p(loss), p(counts), p(mean),
                                        p(ws), nbytes, st))
        gpu_lib._check(L.mx_moe_balance_bwd(p(z), 0, p(bias), p(counts), p(dl), None, p(seg), 3, 2000, 60, 6, None,
                                            p(dz), st))
    side.synchronize()
    assert all(canaries_intact(b) for b, _ in bufs)
    assert all(torch.equal(a, b) for a, b in zip((loss, counts, mean, dz), (*want, wz)))
    got = gpu_lib.mx_moe_balance(z, idx, bias=bias, segments=seg, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    loss, counts, mean = gpu_lib.mx_moe_balance(z[:0], idx[:0], segments=_dev([0, 0, 0]))
    assert not loss.any() and not counts.any() and not mean.any() and counts.shape == (2, 60)
    assert gpu_lib.mx_moe_balance_bwd(z[:0], counts, 6, dloss=dl[:2], segments=_dev([0, 0, 0])).shape == (0, 60)


def test_two_graphs_that_share_a_workspace(gpu_lib):
    """Forward and backward captured twice over one workspace, replayed several
    times with new inputs and eager calls in between."""
    T, E, k = 1500, 16, 2
    ws = torch.empty(gpu_lib.moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    dl = torch.full((1,), 0.5, device="cuda")
    sets = [_inputs(gpu_lib, T, E, k, torch.float32, 20 + i)[::2] for i in range(2)]
    outs, graphs = [], []

    def run(z, idx, w):
        loss, counts, mean = gpu_lib.mx_moe_balance(z, idx, workspace=w)
        return loss, counts, mean, gpu_lib.mx_moe_balance_bwd(z, counts, k, dloss=dl)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*sets[0], ws)
    torch.cuda.current_stream().wait_stream(side)
    for z, idx in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(z, idx, ws))
        graphs.append(g)
    for turn in range(4):
        for (z, idx), out, g in zip(sets, outs, graphs):
            z.copy_(torch.randn_like(z) * (1 + turn))
            idx.copy_(gpu_lib.mx_moe_route(z, k)[0])
            g.replay()
            want = run(z, idx, None)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_with_the_routers_gradient(gpu_lib):
    """A training step's router: choices, weights, balance loss; the gradient of
    both from one array, against 64 bits."""
    T, E, k = 700, 8, 2
    z, bias, _ = _inputs(gpu_lib, T, E, k, torch.float32, 9, masked=False)
    zz = z.clone().requires_grad_()
    idx, w = gpu_lib.MoERoute.apply(zz, k, bias, True)
    loss, counts, _ = gpu_lib.MoEBalance.apply(zz, idx, bias, None)
    dw = torch.randn((T, k), device="cuda") * 1e-3
    ((w * dw).sum() + 0.01 * loss.sum()).backward()
    i, wt, lse = gpu_lib.mx_moe_route(z, k, bias=bias)
    dz = gpu_lib.mx_moe_route_bwd(z, i, wt, lse, dw, bias=bias)
    gpu_lib.mx_moe_balance_bwd(z, counts, k, dloss=torch.full((1,), 0.01, device="cuda"), bias=bias, add=dz, out=dz)
    z64 = z.double().cpu().requires_grad_()
    ek = torch.exp(z64).gather(1, idx.long().cpu())
    c = counts[0].double().cpu()
    total = (ek / ek.sum(1, keepdim=True) * dw.double().cpu()).sum()
    (total + 0.01 * E / (k * T) * (c * torch.softmax(z64, 1).mean(0)).sum()).backward()
    want = z64.grad.numpy()
    # both parts are relative to sizes of at most |dw| and 0.01 E max(c) / (k T^2), with some 64 half steps of fp32
    size = np.abs(dw.cpu().numpy()).sum(1, keepdims=True) + 0.01 * E * float(c.max()) / (k * T * T)
    assert np.all(np.abs(f64(dz) - want) <= 64 * 2.0 ** -24 * size)
    assert np.all(np.abs(f64(zz.grad) - want) <= 64 * 2.0 ** -24 * size)

"""The router (mx_moe_route, mx_moe_route_bwd, MoERoute) against the 64-bit
form: choices exactly, weights, log-sums and gradients within derived bounds;
the training chain route -> dispatch -> grouped MLP -> dprobs -> router
gradient ("Efficient MoE training for biological foundation models", Dense vs.
MoE scaling)."""
import numpy as np
import pytest
import torch

from tests import decode_ref as ref
from tests.gpu_util import canaries_intact, guarded

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1), (1, 8, 2), (3, 4, 4), (7, 5, 2), (33, 8, 8), (64, 16, 16), (65, 17, 3), (300, 60, 6), (129, 64, 16),
          (257, 65, 5), (1000, 128, 8), (31, 127, 16), (4099, 8, 2)]


def _inputs(T, E, dtype, seed, masked=True):
    gen = torch.Generator().manual_seed(seed)
    z = (2 * torch.randn((T, E), generator=gen)).to(dtype)
    if masked:
        z[torch.rand((T, E), generator=gen) < 0.1] = float("-inf")
        if T > 2:
            z[1] = float("-inf")                       # nothing open
            z[2, 1:] = float("-inf")                   # one open
    return z.cuda(), (0.3 * torch.randn(E, generator=gen)).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_choices_weights_and_log_sums(gpu_lib, T, E, k, dtype):
    z, bias = _inputs(T, E, dtype, T + E)
    for renorm in (True, False):
        for b in (None, bias):
            idx, w, lse = gpu_lib.mx_moe_route(z, k, bias=b, renormalize=renorm)
            ri, rw, rl, rel, lb = ref.route(ref.f64(z), None if b is None else b.cpu().numpy(), k, renorm)
            assert idx.dtype == torch.int32 and np.array_equal(idx.cpu().numpy(), ri)
            assert np.all(np.abs(ref.f64(w) - rw) <= rel * rw)
            fin = np.isfinite(rl)
            assert np.array_equal(np.isfinite(ref.f64(lse)), fin)
            assert np.all(np.abs(ref.f64(lse) - rl)[fin] <= lb[fin])


def test_ties_go_to_the_lower_expert(gpu_lib):
    for E, k in ((8, 3), (16, 5), (60, 9), (128, 16)):
        z = torch.zeros((5, E), device="cuda")
        z[1, E // 2:] = 1.0
        z[2, ::3] = 2.0
        z[3] = -torch.finfo(torch.float32).max         # the type's lowest value is a value
        z[4, 1::2] = -0.0                              # equal to 0
        idx, w, _ = gpu_lib.mx_moe_route(z, k)
        ri, rw, _, rel, _ = ref.route(z.cpu().numpy(), None, k, True)
        assert np.array_equal(idx.cpu().numpy(), ri)
        assert np.all(np.abs(ref.f64(w) - rw) <= rel * rw)


def test_nan_and_shut_experts(gpu_lib):
    z = torch.randn((4, 12), device="cuda")
    z[0, 3] = float("nan")
    z[1] = float("nan")
    z[2, :11] = float("-inf")
    bias = torch.zeros(12, device="cuda")
    bias[5], bias[7] = float("-inf"), float("nan")
    z[3, 6] = float("inf")                             # chosen; its weights are unspecified
    idx, w, lse = gpu_lib.mx_moe_route(z, 4, bias=bias)
    i = idx.cpu().numpy()
    assert not np.isin(i, [5, 7]).any() and 3 not in i[0] and (i[1] == -1).all()
    assert list(i[2]) == [11, -1, -1, -1] and i[3, 0] == 6 and len(set(i[3])) == 4
    assert torch.equal(w[1], torch.zeros(4, device="cuda")) and torch.equal(w[2].cpu(), torch.tensor([1.0, 0, 0, 0]))
    assert lse[1] == float("-inf") and torch.isfinite(w[:3]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gradient_against_the_formula(gpu_lib, T, E, k, dtype):
    z, bias = _inputs(T, E, dtype, 7 * T + E)
    rng = np.random.default_rng(T)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    for renorm in (True, False):
        for b in (None, bias):
            idx, w, lse = gpu_lib.mx_moe_route(z, k, bias=b, renormalize=renorm)
            dw[idx < 0] = float("nan")                 # never read as a gradient
            dz = gpu_lib.mx_moe_route_bwd(z, idx, w, lse, dw, bias=b, renormalize=renorm)
            want, bound = ref.route_bwd(ref.f64(z), None if b is None else ref.f64(b), idx.cpu().numpy(), ref.f64(w),
                                        ref.f64(lse), ref.f64(dw), renorm)
            if dtype == torch.bfloat16:
                bound = bound + ref.BF16_HALF * (np.abs(want) + bound)
            got = ref.f64(dz)
            assert dz.dtype == dtype and np.all(np.abs(got - want) <= bound + 1e-37)
            # and through perm: routed rows in another order, some without one
            perm = rng.permutation(T * k).reshape(T, k).astype(np.int32)
            rows = torch.zeros(T * k, device="cuda")
            rows[torch.from_numpy(perm.reshape(-1)).long().cuda()] = dw.reshape(-1)
            perm[0, 0] = -1
            p = torch.from_numpy(perm).cuda()
            dw2 = dw.clone()
            dw2[0, 0] = 0.0
            a = gpu_lib.mx_moe_route_bwd(z, idx, w, lse, rows, perm=p, bias=b, renormalize=renorm)
            c = gpu_lib.mx_moe_route_bwd(z, idx, w, lse, dw2, bias=b, renormalize=renorm)
            assert torch.equal(a, c)


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(gpu_lib, renorm):
    """Central differences of the 64-bit weights: their error is h^2 times a
    third derivative of at most 1 (softmax) plus rounding 2^-52 / h."""
    z, _ = _inputs(6, 10, torch.float32, 5, masked=False)
    k, h = 3, 1e-4
    zn = ref.f64(z)
    c = np.random.default_rng(1).standard_normal((6, k))
    idx, w, lse = gpu_lib.mx_moe_route(z, k, renormalize=renorm)
    got = ref.f64(gpu_lib.mx_moe_route_bwd(z, idx, w, lse, torch.from_numpy(c.astype(np.float32)).cuda(),
                                           renormalize=renorm))
    pick = idx.cpu().numpy()

    def loss(zz):
        e = np.exp(zz)
        ek = np.take_along_axis(e, pick, 1)
        return (ek / (ek if renorm else e).sum(1, keepdims=True) * c).sum(1)

    num = np.stack([(loss(zn + h * np.eye(10)[e]) - loss(zn - h * np.eye(10)[e])) / (2 * h) for e in range(10)], 1)
    size = np.abs(c).sum(1, keepdims=True)
    assert np.all(np.abs(got - num) <= size * (h * h + 2.0 ** -50 / h + 64 * 2.0 ** -23))


def test_guards_empty_and_streams(gpu_lib):
    z, bias = _inputs(37, 60, torch.bfloat16, 3)
    i0, w0, l0 = gpu_lib.mx_moe_route(z, 6, bias=bias)
    L, p = gpu_lib.load(), gpu_lib._ptr
    bufs = [guarded(s, d) for s, d in (((37, 6), torch.int32), ((37, 6), torch.float32), ((37,), torch.float32),
                                       ((37, 60), torch.bfloat16))]
    (b1, idx), (b2, w), (b3, lse), (b4, dz) = bufs
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gpu_lib._check(L.mx_moe_route(p(z), 0, p(bias), 37, 60, 6, 1, p(idx), p(w), p(lse), gpu_lib._stream()))
        gpu_lib._check(L.mx_moe_route_bwd(p(z), 0, p(bias), p(idx), p(w), p(lse), p(w), 37 * 6, None, 37, 60, 6, 0,
                                          p(dz), gpu_lib._stream()))
    side.synchronize()
    assert all(canaries_intact(b) for b, _ in bufs)
    assert torch.equal(idx, i0) and torch.equal(w, w0) and torch.equal(lse, l0)
    i, w, lse = gpu_lib.mx_moe_route(z[:0], 6)
    assert i.shape == (0, 6) and gpu_lib.mx_moe_route_bwd(z[:0], i, w, lse, w).shape == (0, 60)


def test_captured_forward_and_backward(gpu_lib):
    z, _ = _inputs(50, 16, torch.float32, 4)
    dprobs = torch.randn(100, device="cuda")
    perm = torch.randperm(100, device="cuda").to(torch.int32).view(50, 2)

    def step():
        idx, w, lse = gpu_lib.mx_moe_route(z, 2, renormalize=False)
        return idx, w, gpu_lib.mx_moe_route_bwd(z, idx, w, lse, dprobs, perm=perm, renormalize=False)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        z.copy_(_inputs(50, 16, torch.float32, 40 + i)[0])
        want = step()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_autograd_function(gpu_lib):
    for dtype, renorm in ((torch.float32, True), (torch.bfloat16, False)):
        z, bias = _inputs(20, 8, dtype, 9, masked=False)
        z.requires_grad_()
        idx, w = gpu_lib.MoERoute.apply(z, 2, bias, renorm)
        c = torch.randn_like(w)
        (w * c).sum().backward()
        i0, w0, l0 = gpu_lib.mx_moe_route(z.detach(), 2, bias=bias, renormalize=renorm)
        assert torch.equal(idx, i0) and torch.equal(w, w0) and not idx.requires_grad
        assert torch.equal(z.grad, gpu_lib.mx_moe_route_bwd(z.detach(), i0, w0, l0, c, bias=bias, renormalize=renorm))


def test_autograd_function_refuses_a_second_derivative(gpu_lib):
    z, _ = _inputs(5, 8, torch.float32, 10, masked=False)
    z.requires_grad_()
    _, w = gpu_lib.MoERoute.apply(z, 2)
    (g,) = torch.autograd.grad((w * w).sum(), z, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_training_chain(gpu_lib):
    """route -> dispatch -> fused MLP forward and backward -> dprobs -> the
    router's gradient, with tokens that have one open expert, or none."""
    mx = gpu_lib
    gen = torch.Generator().manual_seed(30)
    T, E, k, H, F = 200, 8, 2, 128, 128
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    z, _ = _inputs(T, E, torch.float32, 31)
    w1 = (0.05 * torch.randn((E, 2 * F, H), generator=gen)).to(torch.bfloat16).cuda()
    w2 = (0.05 * torch.randn((E, H, F), generator=gen)).to(torch.bfloat16).cuda()
    idx, w, lse = mx.mx_moe_route(z, k)
    x_perm, probs, perm, row_token, counts = mx.mx_moe_dispatch(x, idx, w, E)
    R = int(counts.sum())
    assert R == int((idx >= 0).sum()) < T * k
    y, st = mx.grouped_mlp_fwd(x_perm[:R].contiguous(), probs[:R].contiguous(), w1, w2, counts.tolist())
    dy = torch.randn((R, H), generator=gen).to(torch.bfloat16).cuda()
    _, dprobs, _, _ = mx.grouped_mlp_bwd(dy, probs[:R].contiguous(), st)
    dz = mx.mx_moe_route_bwd(z, idx, w, lse, dprobs, perm=perm)
    dw = np.zeros((T, k))
    pn = perm.cpu().numpy()
    dw[pn >= 0] = ref.f64(dprobs)[pn[pn >= 0]]
    want, bound = ref.route_bwd(ref.f64(z), None, idx.cpu().numpy(), ref.f64(w), ref.f64(lse), dw, True)
    assert np.all(np.abs(ref.f64(dz) - want) <= bound + 1e-37)
    assert np.abs(want).max() > 0


def test_topk_out_of_range_is_refused_before_anything_is_allocated(gpu_lib):
    z = torch.zeros((64, 8), device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for k in (0, -1, 9, 10 ** 9, 2 ** 32 + 2):
        with pytest.raises(gpu_lib.MXError):
            gpu_lib.mx_moe_route(z, k)
    assert torch.cuda.max_memory_allocated() - before <= 4096

"""8-bit integers (mx_quantize_int8, mx_gemm_int8, mx_grouped_gemm_int8,
grouped_mlp_fwd_int8) against 64 bits: codes and scales exactly, products and the
MLP within derived bounds; odd sizes, strides, empty groups, sizes on the device,
infinities, streams, graphs."""
import numpy as np
import pytest
import torch

from tests import decode_ref
from tests import int8_ref as ref
from tests.gpu_util import canaries_intact, guarded

pytestmark = pytest.mark.gpu

f64 = decode_ref.f64
BF16_HALF = decode_ref.BF16_HALF


def _x(rows, cols, dtype, seed):
    """Values with ties: bf16 rows whose largest value is 127 times a power of two
    put many quotients exactly on a half."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=gen)
    x[:, : cols // 8] *= 8
    for r in range(rows):
        if r % 4 == 1:
            x[r] = torch.randint(-254, 255, (cols,), generator=gen) * 2.0 ** (r % 7 - 3)
            x[r, r % cols] = 254 * 2.0 ** (r % 7 - 3)
        if r % 8 == 3:
            x[r] *= 2.0 ** -90 if r % 16 == 3 else 2.0 ** 100
        if r % 16 == 6:
            x[r] = 0
        if r % 16 == 14:
            x[r] *= 2.0 ** -115                            # below the least top
    return x.to(dtype).cuda()


def _check_cast(q, s, x, weight=None):
    rq, rs = ref.cast(f64(x), None if weight is None else weight.cpu().numpy())
    assert q.dtype == torch.int8 and s.dtype == torch.float32
    assert np.array_equal(q.cpu().numpy().astype(np.int64), rq) and np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 48), (33, 512), (33, 528), (7, 2048), (66, 2064), (33, 4096), (18, 4112),
                                       (9, 16384), (6, 16400), (3, 40000), (1000, 256)])
def test_cast_is_exact(gpu_lib, rows, cols, dtype):
    x = _x(rows, cols, dtype, rows + cols)
    _check_cast(*gpu_lib.mx_quantize_int8(x), x)
    w = torch.randn(rows, device="cuda")
    _check_cast(*gpu_lib.mx_quantize_int8(x, row_weight=w), x, w)
    gen = torch.Generator().manual_seed(rows)
    idx = torch.randint(0, rows, (2 * rows + 1,), generator=gen).to(torch.int32).cuda()
    _check_cast(*gpu_lib.mx_quantize_int8(x, row_index=idx), x[idx.long()])
    wide = torch.full((rows, cols + 24), float("nan"), dtype=dtype, device="cuda")
    wide[:, 16:16 + cols] = x
    _check_cast(*gpu_lib.mx_quantize_int8(wide[:, 16:16 + cols]), x)


def test_every_bf16_tie(gpu_lib):
    """All 128 significands of a row's top against all of a value, a few exponents apart."""
    top = torch.arange(128, 256).float()
    v = torch.cat([torch.arange(128, 256).float() * 2.0 ** e for e in range(-9, 1)])
    x = torch.minimum(v[None], top[:, None]).repeat(1, 2)
    x[:, 1::2] *= -1
    x[:, 0] = top
    x = x.to(torch.bfloat16).cuda()
    _check_cast(*gpu_lib.mx_quantize_int8(x), x)


def test_fp32_values_beside_ties(gpu_lib):
    """fp32 values half a step and a step beside (2 j + 1) top / 254, for many tops."""
    rng = np.random.default_rng(4)
    top = rng.uniform(1, 2, 400).astype(np.float32) * np.float32(2.0) ** rng.integers(-60, 100, 400).astype(np.float32)
    j = np.arange(-127, 127)
    half = ((2 * j + 1) * top.astype(np.float64)[:, None] / 254).astype(np.float32)
    x = np.concatenate([half, np.nextafter(half, np.float32(np.inf)), np.nextafter(half, np.float32(-np.inf))], 1)
    x = np.concatenate([np.clip(x, -top[:, None], top[:, None]), top[:, None] * np.ones((1, 16 - x.shape[1] % 16 + 16), np.float32)], 1)
    x = torch.from_numpy(x[:, : x.shape[1] // 16 * 16].astype(np.float32).copy()).cuda()
    _check_cast(*gpu_lib.mx_quantize_int8(x), x)


def test_cast_of_non_finite_rows_indices_outside_and_3d(gpu_lib):
    x = torch.randn((6, 64), device="cuda")
    clean = gpu_lib.mx_quantize_int8(x)
    x[1, 5], x[3, 7], x[4, 0] = float("nan"), float("inf"), float("-inf")
    q, s = gpu_lib.mx_quantize_int8(x)
    keep = [0, 2, 5]
    assert torch.equal(q[keep], clean[0][keep]) and torch.equal(s[keep], clean[1][keep])
    assert not torch.isfinite(s[[1, 3, 4]]).any()
    y = gpu_lib.mx_gemm_int8(q, s, clean[0], clean[1])
    assert torch.isfinite(y[keep]).all() and not torch.isfinite(y[[1, 3, 4]]).any()
    idx = torch.tensor([2, -1, 6, 5, 2 ** 31 - 1, -(2 ** 31)], dtype=torch.int32, device="cuda")
    q, s = gpu_lib.mx_quantize_int8(x, row_index=idx)
    assert torch.equal(q[[0, 3]], clean[0][[2, 5]]) and not q[[1, 2, 4, 5]].any() and torch.isfinite(s).all()
    q, s = gpu_lib.mx_quantize_int8(x[:0], row_index=idx)
    assert not q.any()
    w = torch.randn((3, 5, 32), device="cuda").to(torch.bfloat16)
    q, s = gpu_lib.mx_quantize_int8(w)
    assert q.shape == (3, 5, 32) and s.shape == (3, 5)
    _check_cast(q.view(15, 32), s.view(15), w.view(15, 32))
    assert gpu_lib.mx_quantize_int8(x[:0])[0].shape == (0, 64)
    assert gpu_lib.mx_quantize_int8(x, row_index=idx[:0], row_weight=x[:0, 0].contiguous())[1].shape == (0,)


def _codes(gen, *shape):
    return torch.randint(-128, 128, shape, generator=gen, dtype=torch.int8).cuda()


def _scales(gen, *shape):
    return (torch.rand(shape, generator=gen) * 0.02 + 0.001).cuda()


def _close(got, want, bound):
    if got.dtype == torch.bfloat16:
        bound = bound + BF16_HALF * (np.abs(want) + bound)
    assert np.all(np.abs(f64(got) - want) <= bound)


SIZES = [(1, 1, 16), (1, 999, 544), (2, 17, 128), (5, 64, 144), (16, 300, 4096), (17, 33, 272), (31, 65, 112), (33, 129, 256),
         (64, 256, 1024), (65, 257, 240), (100, 4096, 512), (129, 31, 2048), (255, 511, 384), (257, 640, 400),
         (1000, 1111, 640), (2049, 2050, 128), (3, 1, 131056)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(gpu_lib, m, n, k):
    gen = torch.Generator().manual_seed(m + n + k)
    a, b = _codes(gen, m, k), _codes(gen, n, k)
    sa, sb = _scales(gen, m), _scales(gen, n)
    want, bound = ref.product(a.cpu().numpy(), sa.cpu().numpy(), b.cpu().numpy(), sb.cpu().numpy())
    for dt in (torch.bfloat16, torch.float32):
        _close(gpu_lib.mx_gemm_int8(a, sa, b, sb, out_dtype=dt), want, bound)


# each kernel form once more at a size that takes it, whole and with k shared out
# over workgroups (those need a workspace): rows per group, n, k
FORMS = [([130], 6000, 64), ([67, 0, 133], 6000, 64), ([200], 6000, 272), ([100, 40, 60], 6000, 272), ([400], 12000, 144),
         ([12], 11500, 144), ([24], 11000, 272), ([1, 300, 99], 12000, 144), ([896, 1409], 16000, 512), ([1000], 4501, 272),
         ([400, 0, 600], 4500, 400), ([400, 0, 600], 4500, 528), ([1000], 4501, 1040), ([400, 0, 600], 4500, 1168),
         ([400, 0, 600], 4500, 1296)]
SHARED = [([130], 100, 8192), ([130], 101, 8192), ([60, 0, 140], 1030, 4112), ([200], 2050, 4112), ([200], 2051, 4112),
          ([130, 170, 100], 6000, 4112), ([3, 0, 0, 5], 48, 16384), ([200], 4500, 8192), ([200], 5120, 13824)]
# ... and for the tiles of the last round alone
TAILS = [([4000], 4300, 4096), ([1000, 0, 3100], 4301, 2064), ([4100], 4096, 4096), ([1920, 2177], 6000, 4096)]


@pytest.mark.parametrize("sizes,n,k", FORMS + SHARED + TAILS)
def test_product_of_each_form(gpu_lib, sizes, n, k):
    gen = torch.Generator().manual_seed(n + k)
    G, m = len(sizes), sum(sizes)
    a, b, sa, sb = _codes(gen, m, k), _codes(gen, G, n, k), _scales(gen, m), _scales(gen, G, n)
    ends = np.cumsum([0] + sizes)
    # sums of integers below 2^53: exact in 64 bits
    want = torch.cat([(a[s:e].double() @ b[g].double().T.contiguous()) * sa[s:e].double()[:, None] * sb[g].double()
                      for g, (s, e) in enumerate(zip(ends[:-1], ends[1:]))]).cpu().numpy()
    nbytes = gpu_lib.gemm_int8_workspace_bytes(m, n, k, G)
    assert (nbytes > 0) == ((sizes, n, k) in SHARED + TAILS)
    counts = torch.tensor(sizes, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        wbuf, ws = guarded((nbytes,), torch.uint8)
        buf, out = guarded((m, n), dt)
        gpu_lib.mx_grouped_gemm_int8(a, sa, b, sb, sizes, out=out, workspace=ws)
        _close(out, want, 3.01 * ref.U * np.abs(want))
        assert canaries_intact(buf) and canaries_intact(wbuf)
        assert torch.equal(out, gpu_lib.mx_grouped_gemm_int8(a, sa, b, sb, counts, out_dtype=dt))
        if G == 1:
            assert torch.equal(out, gpu_lib.mx_gemm_int8(a, sa, b[0], sb[0], out_dtype=dt))
    if nbytes:
        with pytest.raises(gpu_lib.MXError):
            gpu_lib.mx_grouped_gemm_int8(a, sa, b, sb, counts, workspace=ws[:-1])


def test_two_graphs_that_share_a_workspace(gpu_lib):
    """Two products with k shared out, captured over one workspace, replayed in
    turn with new inputs and eager calls in between."""
    gen = torch.Generator().manual_seed(31)
    shapes = [(130, 100, 8192), (64, 300, 8208)]
    ws = torch.empty(max(gpu_lib.gemm_int8_workspace_bytes(*s) for s in shapes), dtype=torch.uint8, device="cuda")
    assert all(gpu_lib.gemm_int8_workspace_bytes(*s) > 0 for s in shapes)
    sets = [(_codes(gen, m, k), _scales(gen, m), _codes(gen, n, k), _scales(gen, n)) for m, n, k in shapes]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gpu_lib.mx_gemm_int8(*sets[0], workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gpu_lib.mx_gemm_int8(*s, workspace=ws))
        graphs.append(g)
    for _ in range(4):
        for s, g, out in zip(sets, graphs, outs):
            s[0].copy_(_codes(gen, *s[0].shape))
            g.replay()
            want = gpu_lib.mx_gemm_int8(*s)
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_largest_sums(gpu_lib):
    """-128 times -128 summed over the longest k stays below 2^31."""
    for m, n in ((1, 3), (40, 70), (300, 300)):
        k = 131056
        a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
        b = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
        c = gpu_lib.mx_gemm_int8(a, torch.ones(m, device="cuda"), b, torch.ones(n, device="cuda"), out_dtype=torch.float32)
        assert torch.equal(c, torch.full((m, n), float(16384 * k), device="cuda"))


GROUPS = [([3], 40, 64), ([0, 5, 0, 1], 33, 128), ([1, 1, 1, 1, 1], 100, 272), ([40, 0, 33, 7], 130, 256),
          ([300, 1, 0, 129, 64], 257, 144), ([0, 0, 700], 512, 512), ([513, 256, 255, 1024], 600, 384), ([2] * 128, 48, 96),
          ([0] * 60 + [77] + [3] * 30, 80, 160)]


@pytest.mark.parametrize("sizes,n,k", GROUPS)
def test_grouped_product(gpu_lib, sizes, n, k):
    gen = torch.Generator().manual_seed(n + k)
    G, m = len(sizes), sum(sizes)
    a, b = _codes(gen, m, k), _codes(gen, G, n, k)
    sa, sb = _scales(gen, m), _scales(gen, G, n)
    ends = np.cumsum([0] + sizes)
    parts = [ref.product(a[s:e].cpu().numpy(), sa[s:e].cpu().numpy(), b[g].cpu().numpy(), sb[g].cpu().numpy())
             for g, (s, e) in enumerate(zip(ends[:-1], ends[1:]))]
    want, bound = np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])
    counts = torch.tensor(sizes, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        host = gpu_lib.mx_grouped_gemm_int8(a, sa, b, sb, sizes, out_dtype=dt)
        _close(host, want, bound)
        assert torch.equal(host, gpu_lib.mx_grouped_gemm_int8(a, sa, b, sb, counts, out_dtype=dt))
    # rows behind the last group are left as they were, also on a call with more rows than groups name
    if m > 2:
        counts[-1] = 0
        left = m - sizes[-1]
        buf, out = guarded((m, n), torch.float32)
        out.fill_(7.0)
        gpu_lib.mx_grouped_gemm_int8(a, sa, b, sb, counts, out=out)
        assert torch.equal(out[:left], host[:left]) and torch.all(out[left:] == 7.0) and canaries_intact(buf)


def test_counts_that_do_not_fit_are_cut(gpu_lib):
    gen = torch.Generator().manual_seed(1)
    m, n, k, G = 50, 40, 64, 5
    a, b, sa, sb = _codes(gen, m, k), _codes(gen, G, n, k), _scales(gen, m), _scales(gen, G, n)
    for counts, cut in (([10, -3, 20, 1000, 5], [10, 0, 20, 20, 0]), ([2 ** 62, 2 ** 62, 1, 1, 1], [50, 0, 0, 0, 0]),
                        ([-(2 ** 63), 2 ** 63 - 1, 0, 0, 0], [0, 50, 0, 0, 0])):
        got = gpu_lib.mx_grouped_gemm_int8(a, sa, b, sb, torch.tensor(counts, device="cuda"), out_dtype=torch.float32)
        assert torch.equal(got, gpu_lib.mx_grouped_gemm_int8(a, sa, b, sb, cut, out_dtype=torch.float32))


def test_guards_streams_and_repeats(gpu_lib):
    gen = torch.Generator().manual_seed(2)
    for m, n, k in ((3, 77, 160), (90, 130, 528), (700, 900, 256)):
        a, b, sa, sb = _codes(gen, m, k), _codes(gen, n, k), _scales(gen, m), _scales(gen, n)
        for dt in (torch.bfloat16, torch.float32):
            buf, out = guarded((m, n), dt)
            want = gpu_lib.mx_gemm_int8(a, sa, b, sb, out_dtype=dt)
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            gpu_lib.mx_gemm_int8(a, sa, b, sb, out=out, stream=side)
            again = gpu_lib.mx_gemm_int8(a, sa, b, sb, out_dtype=dt, stream=side)
            side.synchronize()
            assert canaries_intact(buf) and torch.equal(out, want) and torch.equal(again, want)
    x = torch.randn((33, 528), device="cuda")
    bufs = [guarded((33, 528), torch.int8), guarded((33,), torch.float32)]
    p = gpu_lib._ptr
    gpu_lib._check(gpu_lib.load().mx_quantize_int8(p(x), 1, 33, 528, 528, None, 33, None, p(bufs[0][1]), p(bufs[1][1]),
                                                   gpu_lib._stream()))
    _check_cast(bufs[0][1], bufs[1][1], x)
    assert all(canaries_intact(b) for b, _ in bufs)


def _weights(gpu_lib, gen, E, H, F):
    w1 = (0.05 * torch.randn((E, 2 * F, H), generator=gen)).cuda()
    w2 = (0.05 * torch.randn((E, H, F), generator=gen)).cuda()
    return (*gpu_lib.mx_quantize_int8(w1), *gpu_lib.mx_quantize_int8(w2))


def _mlp_ref(x, probs, w, sizes):
    w1, s1, w2, s2 = (t.cpu().numpy() for t in w)
    ends = np.cumsum([0] + list(sizes))
    out = [ref.mlp(x[s:e], None if probs is None else probs[s:e], w1[g], s1[g], w2[g], s2[g])
           for g, (s, e) in enumerate(zip(ends[:-1], ends[1:])) if e > s]
    return np.concatenate([o[0] for o in out]), np.concatenate([o[1] for o in out])


MLPS = [([70, 0, 60], 8192, 64), ([130], 64, 8192), ([1], 32, 32), ([3, 0, 2], 64, 96), ([0, 40, 1, 33], 96, 160),
        ([130, 0, 257], 256, 224), ([600, 700], 128, 256), ([1] * 16, 288, 64), ([2300], 4096, 3712), ([1500, 0, 2600], 4096, 2176),
        ([400, 0, 600], 288, 2272), ([400, 0, 600], 1056, 2272)]


@pytest.mark.parametrize("sizes,H,F", MLPS)
def test_mlp(gpu_lib, sizes, H, F):
    gen = torch.Generator().manual_seed(H + F)
    E, R = len(sizes), sum(sizes)
    w = _weights(gpu_lib, gen, E, H, F)
    x = torch.randn((R, H), generator=gen).to(torch.bfloat16).cuda()
    probs = torch.rand(R, generator=gen).cuda()
    counts = torch.tensor(sizes, device="cuda")
    for p in (probs, None):
        y = gpu_lib.grouped_mlp_fwd_int8(x, p, *w, sizes)
        _close(y, *_mlp_ref(f64(x), None if p is None else f64(p), w, sizes))
        assert torch.equal(y, gpu_lib.grouped_mlp_fwd_int8(x, p, *w, counts))
    # the same rows through an index into fewer tokens
    token = torch.randint(0, max(1, R // 2), (R,), generator=gen).to(torch.int32).cuda()
    some = x[: max(1, R // 2)].contiguous()
    want = gpu_lib.grouped_mlp_fwd_int8(some[token.long()], probs, *w, sizes)
    nbytes = gpu_lib.mlp_int8_workspace_bytes(E, R, H, F)
    buf, ws = guarded((nbytes,), torch.uint8)
    obuf, out = guarded((R, H), torch.bfloat16)
    got = gpu_lib.grouped_mlp_fwd_int8(some, probs, *w, counts, row_token=token, out=out, workspace=ws)
    assert torch.equal(got, want) and canaries_intact(buf) and canaries_intact(obuf)


def test_mlp_is_its_parts(gpu_lib):
    """The MLP's bits are those of the public casts and products with the SwiGLU in
    between, where the middle agrees to fp32: second product of the same codes."""
    gen = torch.Generator().manual_seed(5)
    sizes, H, F = [50, 30, 0, 90], 128, 192
    w = _weights(gpu_lib, gen, 4, H, F)
    x = torch.randn((170, H), generator=gen).to(torch.bfloat16).cuda()
    probs = torch.rand(170, generator=gen).cuda()
    q, s = gpu_lib.mx_quantize_int8(x)
    h = gpu_lib.mx_grouped_gemm_int8(q, s, w[0], w[1], sizes, out_dtype=torch.float32)
    a = torch.nn.functional.silu(h[:, :F].double()) * h[:, F:].double()
    q, s = gpu_lib.mx_quantize_int8(a.float(), row_weight=probs)
    y = gpu_lib.mx_grouped_gemm_int8(q, s, w[2], w[3], sizes)
    want, bound = _mlp_ref(f64(x), f64(probs), w, sizes)
    _close(y, want, bound)
    _close(gpu_lib.grouped_mlp_fwd_int8(x, probs, *w, sizes), want, bound)


def test_mlp_rows_without_an_expert_and_rows_with_a_nan(gpu_lib):
    gen = torch.Generator().manual_seed(6)
    H, F, R = 64, 96, 80
    w = _weights(gpu_lib, gen, 3, H, F)
    x = torch.randn((R, H), generator=gen).to(torch.bfloat16).cuda()
    y = gpu_lib.grouped_mlp_fwd_int8(x, None, *w, [30, 20, 30])
    counts = torch.tensor([30, 20, 0], device="cuda")
    out = torch.full((R, H), 3.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.grouped_mlp_fwd_int8(x, None, *w, counts, out=out)
    assert torch.equal(out[:50], y[:50]) and torch.all(out[50:] == 3.0)
    x[7, 3], x[40, 0] = float("nan"), float("inf")
    z = gpu_lib.grouped_mlp_fwd_int8(x, None, *w, [30, 20, 30])
    keep = torch.ones(R, dtype=torch.bool)
    keep[[7, 40]] = False
    assert torch.equal(z[keep.cuda()], y[keep.cuda()]) and not torch.isfinite(z[[7, 40]]).any()
    none = gpu_lib.grouped_mlp_fwd_int8(x[:0], None, *w, [0, 0, 0])
    assert none.shape == (0, H)


def test_layer_from_router_to_sum_in_a_graph(gpu_lib):
    """Router, balance, dispatch, MLP over the counts on the device, combine: one
    graph without a wait, replayed with new tokens, each time against 64 bits."""
    gen = torch.Generator().manual_seed(8)
    T, E, k, H, F = 45, 8, 2, 64, 96
    w = _weights(gpu_lib, gen, E, H, F)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    z = torch.randn((T, E), generator=gen).cuda()

    def layer():
        idx, wt, _ = gpu_lib.mx_moe_route(z, k)
        loss, counts, _ = gpu_lib.mx_moe_balance(z, idx)
        _, probs, perm, token, n = gpu_lib.mx_moe_dispatch(x, idx, wt, E, gather=False)
        y = gpu_lib.grouped_mlp_fwd_int8(x, probs, *w, n, row_token=token)
        return gpu_lib.mx_moe_combine(y, perm), loss, counts, n, idx, wt

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer()
    for turn in range(4):
        x.copy_(torch.randn((T, H), generator=gen).to(torch.bfloat16))
        z.copy_(torch.randn((T, E), generator=gen) * (1 + turn))
        g.replay()
        eager = layer()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
        y, _, counts, n, idx, wt = out
        assert torch.equal(counts[0], n)
        # per expert: its tokens in order; the sum of a token's routed rows, each rounded to bf16, rounded again
        i, wn, xn = idx.cpu().numpy(), f64(wt), f64(x)
        total, bound, size = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
        for e in range(E):
            t, j = np.nonzero(i == e)
            if len(t):
                r, b = ref.mlp(xn[t], wn[t, j], *(v[e].cpu().numpy() for v in w))
                np.add.at(total, t, r)
                np.add.at(bound, t, b + BF16_HALF * (np.abs(r) + b))
                np.add.at(size, t, np.abs(r) + b)
        assert np.all(np.abs(f64(y) - total) <= bound + BF16_HALF * (np.abs(total) + bound) + k * 2.0 ** -24 * size)


def test_calls_at_once_on_two_streams(gpu_lib):
    gen = torch.Generator().manual_seed(12)
    sizes, H, F = [40, 25], 128, 128
    w = _weights(gpu_lib, gen, 2, H, F)
    xs = [torch.randn((65, H), generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [gpu_lib.grouped_mlp_fwd_int8(x, None, *w, sizes) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in xs]
    for _ in range(5):
        for x, st, out in zip(xs, streams, got):
            out.append(gpu_lib.grouped_mlp_fwd_int8(x, None, *w, sizes, stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(y, a) for out, a in zip(got, want) for y in out)


def test_binding_refusals(gpu_lib):
    gen = torch.Generator().manual_seed(3)
    a, sa, b, sb = _codes(gen, 4, 32), _scales(gen, 4), _codes(gen, 6, 32), _scales(gen, 6)
    mx = gpu_lib
    for call in (lambda: mx.mx_gemm_int8(a.view(torch.uint8), sa, b, sb), lambda: mx.mx_gemm_int8(a, sa[:3], b, sb),
                 lambda: mx.mx_gemm_int8(a, sa, b[:, :16], sb), lambda: mx.mx_gemm_int8(a, sa, b, sb.double()),
                 lambda: mx.mx_gemm_int8(a, sa, b, sb, out_dtype=torch.float16),
                 lambda: mx.mx_gemm_int8(a, sa, b, sb, out=torch.empty((4, 5), device="cuda")),
                 lambda: mx.mx_grouped_gemm_int8(a, sa, b.view(2, 3, 32), sb.view(2, 3), [1, 2]),
                 lambda: mx.mx_grouped_gemm_int8(a, sa, b.view(2, 3, 32), sb.view(2, 3), [5, -1]),
                 lambda: mx.mx_grouped_gemm_int8(a, sa, b.view(2, 3, 32), sb.view(2, 3), torch.tensor([4, 0], dtype=torch.int32, device="cuda")),
                 lambda: mx.mx_quantize_int8(torch.zeros((32, 4), device="cuda").T),
                 lambda: mx.mx_quantize_int8(torch.zeros((4, 32), device="cuda", dtype=torch.float16)),
                 lambda: mx.mx_quantize_int8(torch.zeros((4, 32), device="cuda"), row_weight=sa[:3]),
                 lambda: mx.mx_quantize_int8(torch.zeros((4, 32), device="cuda"), row_index=torch.zeros(4, dtype=torch.int64, device="cuda")),
                 lambda: mx.mx_quantize_int8(torch.zeros((2, 4, 32), device="cuda"), row_index=torch.zeros(4, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mx.mx_quantize_int8(torch.zeros((4, 24), device="cuda")),
                 lambda: mx.mx_quantize_int8(torch.zeros((4, 33), device="cuda")[:, :32])):
        with pytest.raises(mx.MXError):
            call()

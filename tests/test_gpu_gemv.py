"""Products of a few bf16 rows with 4-bit weights (mx_gemv_fp4, mx_gemv_nvfp4)
against the 64-bit form: bit-exact where every partial sum is exact in fp32,
within the fp32 summation bound otherwise ("TransformerEngine-accelerated
Llama 3 training with native PyTorch training loop", Quantized Training: the
formats)."""
import numpy as np
import pytest
import torch

from tests import decode_ref as ref
from tests.gpu_util import canaries_intact, guarded

pytestmark = pytest.mark.gpu


def _ints(rng, shape, top):
    return rng.integers(-top, top + 1, size=shape).astype(np.float64)


def _bf16(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def _u8(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint8)).cuda()


SIZES = [(1, 1, 32), (1, 16, 32), (1, 17, 64), (2, 33, 96), (3, 250, 160), (1, 999, 544), (7, 64, 2080), (8, 48, 1024),
         (9, 100, 480), (16, 130, 4096), (17, 31, 288), (31, 65, 512), (33, 20, 2336), (48, 80, 352), (64, 100, 704),
         (65, 35, 96), (130, 50, 224), (40, 300, 4096), (64, 129, 7200)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_fp4_integers_are_exact(gpu_lib, m, n, k):
    """Integer rows of at most 8 and scales 2^-1 .. 2^2: every product is a
    multiple of 1/4 and at most 192, so sums below k * 192 <= 2^20 are exact."""
    rng = np.random.default_rng(k * 131 + n * 7 + m)
    x = _ints(rng, (m, k), 8)
    q = rng.integers(0, 256, size=(n, k // 2), dtype=np.uint8)
    s = rng.integers(126, 130, size=(n, k // 32), dtype=np.uint8)
    want = x @ ref.mxfp4(q, s).T
    for dt in (torch.float32, torch.bfloat16):
        buf, out = guarded((m, n), dt)
        got = gpu_lib.mx_gemv_fp4(_bf16(x), _u8(q), _u8(s), out=out)
        torch.cuda.synchronize()
        assert got.data_ptr() == out.data_ptr() and canaries_intact(buf)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.float32).to(dt))


@pytest.mark.parametrize("m,n,k", SIZES)
def test_nvfp4_integers_are_exact(gpu_lib, m, n, k):
    """amax 2688 makes the tensor scale 1; E4M3 scales between 1 and 3.75 in
    steps of 1/8 .. 1/4, so products are multiples of 1/16 and at most 180."""
    rng = np.random.default_rng(k * 137 + n * 5 + m)
    x = _ints(rng, (m, k), 8)
    q = rng.integers(0, 256, size=(n, k // 2), dtype=np.uint8)
    s = rng.integers(0x38, 0x48, size=(n, k // 16), dtype=np.uint8)
    amax = torch.tensor([2688.0], device="cuda")
    want = x @ ref.nvfp4(q, s, 2688.0).T
    for dt in (torch.float32, torch.bfloat16):
        buf, out = guarded((m, n), dt)
        gpu_lib.mx_gemv_nvfp4(_bf16(x), _u8(q), _u8(s), amax, out=out)
        torch.cuda.synchronize()
        assert canaries_intact(buf)
        assert torch.equal(out.cpu(), torch.from_numpy(want).to(torch.float32).to(dt))


@pytest.mark.parametrize("m,n,k", [(17, 70, 8192), (64, 200, 8192), (100, 65, 8192), (16, 50, 8192), (9, 18433, 288),
                                   (16, 18432, 512), (13, 20011, 8192), (8, 18500, 96)])
def test_rows_a_page_apart(gpu_lib, m, n, k):
    """Code rows a multiple of 4096 bytes apart, where workgroups begin at
    places of their own, and many weight rows. Integer rows of at most 4: the products are multiples
    of 1/16 of at most 96, so sums below 8192 * 96 < 2^20 are exact."""
    rng = np.random.default_rng(m + n)
    x = _ints(rng, (m, k), 4)
    q = rng.integers(0, 256, size=(n, k // 2), dtype=np.uint8)
    s4 = rng.integers(126, 130, size=(n, k // 32), dtype=np.uint8)
    sn = rng.integers(0x38, 0x48, size=(n, k // 16), dtype=np.uint8)
    got = gpu_lib.mx_gemv_fp4(_bf16(x), _u8(q), _u8(s4), out_dtype=torch.float32)
    assert np.array_equal(ref.f64(got), x @ ref.mxfp4(q, s4).T)
    got = gpu_lib.mx_gemv_nvfp4(_bf16(x), _u8(q), _u8(sn), torch.tensor([2688.0], device="cuda"), out_dtype=torch.float32)
    assert np.array_equal(ref.f64(got), x @ ref.nvfp4(q, sn, 2688.0).T)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n,k", [(1, 384, 4096), (5, 200, 1568), (40, 96, 2048)])
def test_quantized_weights_within_the_summation_bound(gpu_lib, fmt, m, n, k):
    gen = torch.Generator().manual_seed(m + n + k)
    x = torch.randn((m, k), generator=gen).to(torch.bfloat16)
    w = (0.02 * torch.randn((n, k), generator=gen)).to(torch.bfloat16).cuda()
    if fmt == "mxfp4":
        q, s = gpu_lib.mx_quantize_fp4(w)
        wv = ref.mxfp4(q.cpu().numpy(), s.cpu().numpy())
        call = lambda dt: gpu_lib.mx_gemv_fp4(x.cuda(), q, s, out_dtype=dt)  # noqa: E731
    else:
        q, s, amax = gpu_lib.mx_quantize_nvfp4(w)
        wv = ref.nvfp4(q.cpu().numpy(), s.cpu().numpy(), float(amax))
        call = lambda dt: gpu_lib.mx_gemv_nvfp4(x.cuda(), q, s, amax, out_dtype=dt)  # noqa: E731
    for dt in (torch.float32, torch.bfloat16):
        want, bound = ref.products(ref.f64(x), wv, dt == torch.bfloat16)
        # NVFP4's factor 1/S is one more fp32 product of an fp32 factor
        bound = bound + (2.0 ** -22 * np.abs(want) if fmt == "nvfp4" else 0.0)
        got = ref.f64(call(dt))
        assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / bound)


@pytest.mark.parametrize("first", range(0, 255, 51))
def test_every_fp4_code_and_scale(gpu_lib, first):
    """Unit rows pick single weights: all 16 codes under the E8M0 scale codes
    0 .. 254, subnormal values included, exactly (6 * 2^127 and 4 * 2^127 and
    their like pass fp32's range and are infinite)."""
    scales = np.arange(first, min(first + 51, 255))
    n = len(scales)
    nib = np.tile(np.arange(16, dtype=np.uint8), 2)
    q = np.tile((nib[0::2] | (nib[1::2] << 4))[None], (n, 1))
    x = np.eye(32)[:16]
    got = ref.f64(gpu_lib.mx_gemv_fp4(_bf16(x), _u8(q), _u8(scales[:, None]), out_dtype=torch.float32))
    want = ref.mxfp4(q, scales[:, None])[:, :16].T
    with np.errstate(over="ignore"):
        want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)
    # an infinite weight times the zeros of the other unit rows is NaN there: compare its own place only
    fine = np.isfinite(want).all(0)
    assert np.array_equal(got[:, fine], want[:, fine])
    assert fine.sum() >= n - 2


def test_rows_apart_and_aligned_views(gpu_lib):
    """x as every third row of a wider matrix, from an offset."""
    rng = np.random.default_rng(3)
    m, n, k = 6, 70, 160
    wide = _ints(rng, (3 * m, k + 72), 8)
    q = rng.integers(0, 256, size=(n, k // 2), dtype=np.uint8)
    s = rng.integers(126, 130, size=(n, k // 32), dtype=np.uint8)
    x = _bf16(wide)[1::3, 8:8 + k]
    got = gpu_lib.mx_gemv_fp4(x, _u8(q), _u8(s), out_dtype=torch.float32)
    assert np.array_equal(ref.f64(got), wide[1::3, 8:8 + k] @ ref.mxfp4(q, s).T)


def test_nonfinite_rows_stay_apart(gpu_lib):
    rng = np.random.default_rng(4)
    for m in (3, 20):
        x = _ints(rng, (m, 96), 4)
        q = rng.integers(0, 256, size=(40, 48), dtype=np.uint8)
        s = np.full((40, 3), 127, dtype=np.uint8)
        clean = gpu_lib.mx_gemv_fp4(_bf16(x), _u8(q), _u8(s))
        bad = x.copy()
        bad[1, 5], bad[2, 95] = np.nan, np.inf
        got = gpu_lib.mx_gemv_fp4(_bf16(bad), _u8(q), _u8(s))
        keep = [r for r in range(m) if r not in (1, 2)]
        assert torch.equal(got[keep], clean[keep])
        assert torch.isnan(got[1]).all()


def test_empty_and_zero_weights(gpu_lib):
    q, s = torch.zeros((5, 16), dtype=torch.uint8, device="cuda"), torch.zeros((5, 1), dtype=torch.uint8, device="cuda")
    assert gpu_lib.mx_gemv_fp4(torch.zeros((0, 32), dtype=torch.bfloat16, device="cuda"), q, s).shape == (0, 5)
    assert gpu_lib.mx_gemv_fp4(torch.ones((2, 32), dtype=torch.bfloat16, device="cuda"), q[:0], s[:0]).shape == (2, 0)
    y = gpu_lib.mx_gemv_nvfp4(torch.ones((2, 32), dtype=torch.bfloat16, device="cuda"), q,
                              torch.zeros((5, 2), dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda"))
    assert torch.equal(y, torch.zeros_like(y))


def test_codes_past_four_gib(gpu_lib):
    """n * k / 2 > 2^32 bytes of codes: the last rows are read where they are."""
    n, k = 1 << 19, 16416
    q = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    assert q.numel() > 1 << 32
    s = torch.full((n, k // 32), 127, dtype=torch.uint8, device="cuda")
    q[-3:] = 0x22                                           # 1.0 everywhere
    x = torch.zeros((1, k), dtype=torch.bfloat16, device="cuda")
    x[0, ::19] = 1.0
    y = gpu_lib.mx_gemv_fp4(x, q, s, out_dtype=torch.float32)[0]
    ones = len(range(0, k, 19))
    assert torch.equal(y[-3:].cpu(), torch.full((3,), float(ones))) and int((y != 0).sum()) == 3


def test_repeats_bit_for_bit_on_streams_and_in_graphs(gpu_lib):
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((4, 1024), generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.randn((300, 1024), generator=gen, device="cuda").to(torch.bfloat16)
    q, s = gpu_lib.mx_quantize_fp4(w)
    out = torch.empty((4, 300), dtype=torch.float32, device="cuda")
    want = gpu_lib.mx_gemv_fp4(x, q, s, out_dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gpu_lib.mx_gemv_fp4(x, q, s, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.mx_gemv_fp4(x, q, s, out=out)
    for i in range(4):
        x.copy_(torch.randn((4, 1024), generator=gen, device="cuda"))
        eager = gpu_lib.mx_gemv_fp4(x, q, s, out_dtype=torch.float32)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


def test_every_nvfp4_code_and_scale(gpu_lib):
    """Unit rows pick single weights: all 16 codes under every E4M3 scale, the
    subnormal ones and 448 among them, exactly (amax 2688: tensor scale 1)."""
    scales = np.arange(127, dtype=np.uint8)
    q = np.tile(np.tile(np.arange(16, dtype=np.uint8), 2)[0::2] | (np.tile(np.arange(16, dtype=np.uint8), 2)[1::2] << 4), (127, 1))
    s = np.repeat(scales[:, None], 2, axis=1)
    want = ref.nvfp4(q, s, 2688.0).T
    for m in (4, 8, 16, 32):
        got = gpu_lib.mx_gemv_nvfp4(_bf16(np.eye(32)[:m]), _u8(q), _u8(s), torch.tensor([2688.0], device="cuda"),
                                    out_dtype=torch.float32)
        assert np.array_equal(ref.f64(got), want[:m])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n,k", [(40, 300, 4096), (64, 129, 7200), (17, 70, 8192)])
def test_split_products_repeat_in_a_workspace_of_their_size(gpu_lib, fmt, m, n, k):
    """Products that split k over workgroups: the caller's workspace of exactly
    the size asked for, full of NaN before each call; other streams, two graphs
    that share it, replays with new rows and eager work in between."""
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    x = torch.randn((m, k), generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.randn((n, k), generator=gen, device="cuda").to(torch.bfloat16)
    gemv, weight = ((gpu_lib.mx_gemv_fp4, gpu_lib.mx_quantize_fp4(w)) if fmt == "mxfp4" else
                    (gpu_lib.mx_gemv_nvfp4, gpu_lib.mx_quantize_nvfp4(w)))
    nbytes = gpu_lib.gemv_workspace_bytes(m, n, k)
    assert nbytes > 0 and nbytes % (m * n * 4) == 0
    buf, ws = guarded((nbytes,))
    side = torch.cuda.Stream()
    outs, graphs = [torch.empty((m, n), dtype=dt, device="cuda") for dt in (torch.float32, torch.bfloat16)], []
    wants = [gemv(x, *weight, out_dtype=o.dtype) for o in outs]
    for o, want in zip(outs, wants):
        for stream in (None, side):
            ws.fill_(0xFF)
            o.zero_()
            torch.cuda.synchronize()
            gemv(x, *weight, out=o, workspace=ws, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(o, want) and canaries_intact(buf)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gemv(x, *weight, out=o, workspace=ws)
        graphs.append(g)
    with pytest.raises(gpu_lib.MXError):
        gemv(x, *weight, out=outs[0], workspace=ws[:-1])
    for i in range(4):
        x.copy_(torch.randn((m, k), generator=gen, device="cuda"))
        eager = [gemv(x, *weight, out_dtype=o.dtype) for o in outs]
        ws.fill_(0xFF)
        for g, o, want in zip(graphs, outs, eager):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want) and canaries_intact(buf), i

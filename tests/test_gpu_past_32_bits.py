"""Arrays of more than 2^32 elements in the balance loss, the 8-bit integer cast
and the products: what lies on both sides of 2^31 and 2^32, and last."""
import numpy as np
import pytest
import torch

from tests import balance_ref, decode_ref
from tests import int8_ref as ref

pytestmark = pytest.mark.gpu

f64 = decode_ref.f64


@pytest.fixture(autouse=True)
def _memory(gpu_lib):
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB of device memory")
    yield
    torch.cuda.empty_cache()


def test_cast(gpu_lib):
    rows, cols = 70000, 65536
    gen = torch.Generator(device="cuda").manual_seed(1)
    at = [0, 32767, 32768, 65535, 65536, rows - 1]
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[at] = torch.randn((len(at), cols), generator=gen, device="cuda").to(torch.bfloat16)
    q, s = gpu_lib.mx_quantize_int8(x)
    rq, rs = ref.cast(f64(x[at]))
    assert np.array_equal(q[at].cpu().numpy(), rq) and np.array_equal(s[at].cpu().numpy(), rs)
    beside = [1, 32766, 32769, 65534, 65537, rows - 2]
    assert not q[beside].any() and torch.all(s[beside] == np.float32(ref.LEAST) / np.float32(127))
    idx = torch.tensor(at[::-1] + [rows], dtype=torch.int32, device="cuda")
    q, s = gpu_lib.mx_quantize_int8(x, row_index=idx)
    assert np.array_equal(q[:-1].cpu().numpy(), rq[::-1]) and np.array_equal(s[:-1].cpu().numpy(), rs[::-1])
    assert not q[-1].any()


def _codes(gen, *shape):
    return torch.randint(-128, 128, shape, generator=gen, dtype=torch.int8, device="cuda")


def _scales(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda") * 0.02 + 0.001


def _close(got, a, sa, b, sb):
    want, bound = ref.product(*(t.cpu().numpy() for t in (a, sa, b, sb)))
    if got.dtype == torch.bfloat16:
        bound = bound + decode_ref.BF16_HALF * (np.abs(want) + bound)
    assert np.all(np.abs(f64(got) - want) <= bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [65600, 65601])
def test_results(gpu_lib, n, dtype):
    m, k = 70000, 16
    gen = torch.Generator(device="cuda").manual_seed(n)
    a, sa, b, sb = _codes(gen, m, k), _scales(gen, m), _codes(gen, n, k), _scales(gen, n)
    c = gpu_lib.mx_gemm_int8(a, sa, b, sb, out_dtype=dtype)
    for r in (0, 2 ** 31 // n, 2 ** 31 // n + 1, 2 ** 32 // n, 2 ** 32 // n + 1, m - 1):
        _close(c[r:r + 1], a[r:r + 1], sa[r:r + 1], b, sb)


def test_rows(gpu_lib):
    m, n, k = 300000, 40, 16384
    gen = torch.Generator(device="cuda").manual_seed(2)
    a, sa, b, sb = _codes(gen, m, k), _scales(gen, m), _codes(gen, n, k), _scales(gen, n)
    c = gpu_lib.mx_gemm_int8(a, sa, b, sb, out_dtype=torch.float32)
    for r in (0, 2 ** 31 // k - 1, 2 ** 32 // k - 1, m - 3):
        _close(c[r:r + 3], a[r:r + 3], sa[r:r + 3], b, sb)


@pytest.mark.parametrize("sizes", [[3, 0, 2, 0, 4], [30, 0, 41, 3, 70], [300, 0, 290, 30, 400]])
def test_weights(gpu_lib, sizes):
    G, n, k, m = len(sizes), 60000, 16384, sum(sizes)
    gen = torch.Generator(device="cuda").manual_seed(3)
    a, sa, b, sb = _codes(gen, m, k), _scales(gen, m), _codes(gen, G, n, k), _scales(gen, G, n)
    c = gpu_lib.mx_grouped_gemm_int8(a, sa, b, sb, sizes)
    ends = np.cumsum([0] + sizes)
    for g, (s, e) in enumerate(zip(ends[:-1], ends[1:])):
        for n0 in (0, n - 20):
            if e > s:
                _close(c[e - 2:e, n0:n0 + 20], a[e - 2:e], sa[e - 2:e], b[g, n0:n0 + 20], sb[g, n0:n0 + 20])


def test_balance(gpu_lib):
    T, E, k = 33600000, 128, 2
    gen = torch.Generator(device="cuda").manual_seed(4)
    z = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    idx[:, 1] = 1
    o = [0, 16777000, 16777400, 33554200, 33554600, T - 100, T]
    own = [1, 3, 5]                                        # short sequences around 2^31 and 2^32 values, and the last
    for s in own:
        b, e = o[s], o[s + 1]
        z[b:e] = torch.randn((e - b, E), generator=gen, device="cuda").to(torch.bfloat16)
        idx[b:e] = gpu_lib.mx_moe_route(z[b:e], k)[0]
    seg = torch.tensor(o, dtype=torch.int32, device="cuda")
    loss, counts, mean = gpu_lib.mx_moe_balance(z, idx, segments=seg)
    dl, dm = torch.rand(6, generator=gen, device="cuda"), torch.randn((6, E), generator=gen, device="cuda")
    dz = gpu_lib.mx_moe_balance_bwd(z, counts, k, dloss=dl, dmean_prob=dm, segments=seg)
    for s in own:
        b, e = o[s], o[s + 1]
        zn = f64(z[b:e])
        rl, rc, rm, bl, bm = balance_ref.balance(zn, None, idx[b:e].cpu().numpy(), None, E)
        assert np.array_equal(counts[s].cpu().numpy(), rc[0])
        assert np.all(np.abs(f64(mean[s]) - rm[0]) <= bm[0]) and abs(loss[s].item() - rl[0]) <= bl[0]
        want, bound = balance_ref.balance_bwd(zn, None, rc, k, f64(dl[s:s + 1]), f64(dm[s:s + 1]), None, None)
        bound = bound + decode_ref.BF16_HALF * (np.abs(want) + bound)
        assert np.all(np.abs(f64(dz[b:e]) - want) <= bound + 1e-37)
    for s in (0, 2, 4):                                    # even probabilities; two experts take all choices
        n = o[s + 1] - o[s]
        assert counts[s, 0] == counts[s, 1] == n and not counts[s, 2:].any()
        assert torch.all(mean[s] == 1 / E) and loss[s] == 1

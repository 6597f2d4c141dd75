"""Every kernel of the 8-bit integer products (tests/int8_forms.py: its sizes are
checked against the library's plan without a GPU) against 64 bits: results in
bf16 and fp32, rows per group on the host and on the device, and the MLP."""
import numpy as np
import pytest
import torch

from tests import decode_ref
from tests import int8_forms as forms
from tests import int8_ref as ref
from tests.gpu_util import canaries_intact, guarded

pytestmark = pytest.mark.gpu

f64 = decode_ref.f64


def _close(got, want, bound):
    if got.dtype == torch.bfloat16:
        bound = bound + decode_ref.BF16_HALF * (np.abs(want) + bound)
    assert np.all(np.abs(f64(got) - want) <= bound)


@pytest.mark.parametrize("plan,sizes,n,k", forms.PLAIN)
def test_product(gpu_lib, plan, sizes, n, k):
    G, m = len(sizes), sum(sizes)
    assert tuple(gpu_lib.gemm_int8_plan(m, n, k, G, sizes)) == plan
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    a, b = (torch.randint(-128, 128, s, generator=gen, dtype=torch.int8, device="cuda") for s in ((m, k), (G, n, k)))
    sa, sb = (torch.rand(s, generator=gen, device="cuda") * 0.02 + 0.001 for s in ((m,), (G, n)))
    ends = np.cumsum([0] + sizes)
    # sums of integers below 2^53: exact in 64 bits; rounded to fp32 and multiplied twice
    want = torch.cat([(a[s:e].double() @ b[g].double().T.contiguous()) * sa[s:e].double()[:, None] * sb[g].double()
                      for g, (s, e) in enumerate(zip(ends[:-1], ends[1:]))]).cpu().numpy()
    nbytes = gpu_lib.gemm_int8_workspace_bytes(m, n, k, G)
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


@pytest.mark.parametrize("plan,sizes,n,k", forms.SWIGLU)
def test_mlp(gpu_lib, plan, sizes, n, k):
    E, R, H, F = len(sizes), sum(sizes), k, n // 2
    assert tuple(gpu_lib.gemm_int8_plan(R, n, k, E, sizes, swiglu=True)) == plan
    gen = torch.Generator(device="cuda").manual_seed(H + F)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda")
    w1, s1 = gpu_lib.mx_quantize_int8(0.05 * draw(E, 2 * F, H))
    w2, s2 = gpu_lib.mx_quantize_int8(0.05 * draw(E, H, F))
    x, probs = draw(R, H).to(torch.bfloat16), torch.rand(R, generator=gen, device="cuda")
    buf, ws = guarded((gpu_lib.mlp_int8_workspace_bytes(E, R, H, F),), torch.uint8)
    y = gpu_lib.grouped_mlp_fwd_int8(x, probs, w1, s1, w2, s2, sizes, workspace=ws)
    assert canaries_intact(buf)
    counts = torch.tensor(sizes, device="cuda")
    assert torch.equal(y, gpu_lib.grouped_mlp_fwd_int8(x, probs, w1, s1, w2, s2, counts))
    ends = np.cumsum([0] + sizes)
    for g, (s, e) in enumerate(zip(ends[:-1], ends[1:])):
        if e > s:
            w = (t[g].cpu().numpy() for t in (w1, s1, w2, s2))
            _close(y[s:e], *ref.mlp(f64(x[s:e]), f64(probs[s:e]), *w))

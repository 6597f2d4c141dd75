"""How 8-bit integer products run (mx_gemm_int8_plan), without a GPU: the sizes that
the GPU tests run take the kernels they are meant for, and all kernels are among
them; refusals."""
import ctypes
import os

import pytest

import mxfp8_block_scaled_mx_amd as mx
from tests import int8_forms as forms

OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE, EHIP, EUNSUPPORTED = range(7)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mx.lib_path()):
        pytest.skip("library not built")
    return mx.load()


@pytest.mark.parametrize("swiglu", [False, True])
def test_sizes_take_their_kernels(L, swiglu):
    table = forms.SWIGLU if swiglu else forms.PLAIN
    for plan, sizes, n, k in table:
        G, m = len(sizes), sum(sizes)
        host = mx.gemm_int8_plan(m, n, k, G, sizes, swiglu)
        assert tuple(host) == plan, (sizes, n, k)
        if G == 1:
            assert tuple(mx.gemm_int8_plan(m, n, k, swiglu=swiglu)) == plan, (sizes, n, k)
        # sizes on the device: the same, and a last round where any split may have one
        device = mx.gemm_int8_plan(m, n, k, G, None, swiglu)
        assert device[:5] + device[6:] == host[:5] + host[6:] and device.last_round >= host.last_round
        # the workspace is that of the sums
        if not swiglu:
            nbytes = mx.gemm_int8_workspace_bytes(m, n, k, G)
            assert (nbytes >= host.k_parts * m * n * 4) if host.k_parts > 1 else (nbytes > 0) >= host.last_round
    assert {forms.kind(plan, k) for plan, _, _, k in table} == forms.kinds(swiglu)


def test_plan_refusals(L):
    out = (ctypes.c_int32 * 7)()
    sizes = (ctypes.c_int64 * 2)(2, 3)

    def run(m=5, n=64, k=64, G=2, sz=sizes, swiglu=0, p=ctypes.byref(out)):
        return L.mx_gemm_int8_plan(m, n, k, G, sz, swiglu, p)

    assert run() == run(sz=None) == run(swiglu=1) == OK
    assert run(p=None) == run(G=0) == EINVAL
    assert run(m=6) == run(m=-1, sz=None) == run(k=0) == run(k=24) == run(n=-1) == run(n=33, swiglu=1) == ESHAPE
    assert run(G=129, sz=None) == run(n=(1 << 30) + 1) == run(k=131072) == EUNSUPPORTED
    assert run(m=0, G=1, sz=None) == OK and list(out) == [0] * 7
    with pytest.raises(ValueError):
        mx.gemm_int8_plan(5, 64, 64, 2, [5])

"""Refusals of the balance loss and the 8-bit integer calls, without a GPU: bad
arguments get the documented status before anything is enqueued, and the
Python binding refuses tensors that do not fit."""
import ctypes
import os

import pytest
import torch

import mxfp8_block_scaled_mx_amd as mx

OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE, EHIP, EUNSUPPORTED = range(7)
FAKE = ctypes.c_void_p(0x100000)       # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x100001)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mx.lib_path()):
        pytest.skip("library not built")
    return mx.load()


def test_balance_refusals(L):
    n = ctypes.c_size_t()
    assert L.mx_moe_balance_sizes(33, 128, 1, ctypes.byref(n)) == OK and n.value == 0
    assert L.mx_moe_balance_sizes(4096, 8, 1, ctypes.byref(n)) == OK and n.value >= 64 * 8 * 12
    need = n.value
    assert L.mx_moe_balance_sizes(4096, 8, 0, None) == ESHAPE and L.mx_moe_balance_sizes(-1, 8, 1, None) == ESHAPE
    assert L.mx_moe_balance_sizes(4096, 129, 1, None) == L.mx_moe_balance_sizes(4096, 8, 65535, None) == EUNSUPPORTED

    def fwd(z=FAKE, dt=1, b=None, idx=FAKE, seg=None, S=1, T=4096, E=8, k=2, loss=FAKE, c=FAKE, m=FAKE, ws=FAKE, nb=need):
        return L.mx_moe_balance(z, dt, b, idx, seg, S, T, E, k, loss, c, m, ws, nb, None)

    def bwd(z=FAKE, dt=1, b=None, c=FAKE, dl=FAKE, dm=None, seg=None, S=1, T=9, E=8, k=2, add=None, dz=FAKE):
        return L.mx_moe_balance_bwd(z, dt, b, c, dl, dm, seg, S, T, E, k, add, dz, None)

    for f in (fwd, bwd):
        assert f(dt=2) == f(dt=-1) == EINVAL
        assert f(T=-1) == f(E=0) == f(k=0) == f(k=9) == f(S=0) == f(S=-1) == f(S=2) == f(seg=FAKE, S=0) == ESHAPE
        assert f(E=129, k=2) == f(E=128, k=17) == f(T=1 << 27) == f(seg=FAKE, S=65535) == EUNSUPPORTED
        assert f(z=None) == EINVAL
        assert f(z=ODD) == f(b=ODD) == f(c=ODD) == f(seg=ODD) == EALIGN
    assert fwd(idx=None) == fwd(loss=None) == fwd(c=None) == fwd(m=None) == fwd(ws=None) == EINVAL
    assert fwd(idx=ODD) == fwd(loss=ODD) == fwd(m=ODD) == fwd(ws=ctypes.c_void_p(0x100010)) == EALIGN
    assert fwd(nb=need - 1) == EWORKSPACE
    assert bwd(dz=None) == bwd(c=None) == EINVAL
    assert bwd(dl=ODD) == bwd(dm=ODD) == bwd(add=ODD) == bwd(dz=ODD) == EALIGN
    assert bwd(T=0, z=None, dz=None) == OK


def test_cast_refusals(L):
    def run(x=FAKE, dt=0, xr=5, cols=64, ldx=64, idx=None, rows=5, w=None, q=FAKE, s=FAKE):
        return L.mx_quantize_int8(x, dt, xr, cols, ldx, idx, rows, w, q, s, None)

    assert run(dt=2) == run(x=None) == run(q=None) == run(s=None) == EINVAL
    assert run(cols=0) == run(cols=8) == run(cols=-16) == run(xr=-1) == run(rows=-1) == run(rows=4) == ESHAPE
    assert run(ldx=63) == run(ldx=56) == run(ldx=68) == run(dt=1, ldx=66) == run(ldx=-64) == ESHAPE
    assert run(x=ODD) == run(q=ODD) == run(s=ODD) == run(idx=ODD) == run(w=ODD) == EALIGN
    assert run(xr=1 << 24, rows=1 << 24) == run(idx=FAKE, xr=1 << 31) == EUNSUPPORTED
    assert run(cols=(1 << 24) + 16, ldx=1 << 25) == run(ldx=(1 << 24) + 8) == EUNSUPPORTED
    assert run(xr=0, rows=0, x=None) == run(idx=FAKE, rows=0) == OK


def test_product_refusals(L):
    def one(a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, m=5, n=7, k=64, c=FAKE, dt=0, ws=None, nb=0):
        return L.mx_gemm_int8(a, sa, b, sb, m, n, k, c, dt, ws, nb, None)

    sizes = (ctypes.c_int64 * 2)(2, 3)

    def many(a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, m=5, n=7, k=64, c=FAKE, dt=0, sz=sizes, G=2, ws=None, nb=0):
        return L.mx_grouped_gemm_int8(a, sa, b, sb, sz, G, m, n, k, c, dt, ws, nb, None)

    def dev(a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, m=5, n=7, k=64, c=FAKE, dt=0, sz=FAKE, G=2, ws=None, nb=0):
        return L.mx_grouped_gemm_int8_device_split(a, sa, b, sb, sz, G, m, n, k, c, dt, ws, nb, None)

    for f in (one, many, dev):
        assert f(a=None) == f(sa=None) == f(b=None) == f(sb=None) == f(c=None) == f(dt=3) == EINVAL
        assert f(k=0) == f(k=8) == f(k=-16) == f(k=40) == f(n=-1) == ESHAPE
        assert f(n=(1 << 30) + 1) == f(k=131072) == EUNSUPPORTED
        assert f(a=ODD) == f(b=ODD) == f(sa=ODD) == f(sb=ODD) == f(c=ODD) == EALIGN
        assert f(n=0, b=None) == OK
    assert one(m=-1) == ESHAPE and one(m=(1 << 30) + 1) == EUNSUPPORTED and one(m=0, a=None) == OK
    assert one(m=1 << 30, n=1 << 30) == EUNSUPPORTED
    # a product that shares k out over workgroups needs its planes
    n = ctypes.c_size_t()
    assert L.mx_gemm_int8_sizes(16, 4096, 4096, 1, ctypes.byref(n)) == OK and n.value == 0
    big = dict(m=64, n=4096, k=14336)
    assert L.mx_gemm_int8_sizes(*big.values(), 1, ctypes.byref(n)) == OK and n.value % (64 * 4096 * 4) == 0 and n.value > 0
    assert one(**big) == one(**big, nb=n.value) == EINVAL
    assert one(**big, ws=FAKE, nb=n.value - 1) == EWORKSPACE
    assert one(**big, ws=ctypes.c_void_p(0x100010), nb=n.value) == EALIGN
    assert L.mx_gemm_int8_sizes(-1, 1, 16, 1, None) == L.mx_gemm_int8_sizes(1, 1, 24, 1, None) == ESHAPE
    assert L.mx_gemm_int8_sizes(1, 1, 16, 0, None) == EINVAL and L.mx_gemm_int8_sizes(1, 1, 16, 129, None) == EUNSUPPORTED
    assert many(m=6) == many(sz=(ctypes.c_int64 * 2)(-1, 6)) == ESHAPE
    assert many(sz=None) == many(G=0) == dev(sz=None) == dev(G=0) == EINVAL
    assert many(G=129) == dev(G=129) == EUNSUPPORTED
    assert dev(sz=ctypes.c_void_p(0x100004)) == EALIGN
    assert dev(m=-1) == ESHAPE and dev(m=0, a=None) == OK


def test_mlp_refusals(L):
    n = ctypes.c_size_t()

    def size(E=4, R=6, H=64, F=96):
        return L.grouped_mlp_int8_sizes(ctypes.byref(mx._Dims(E, R, H, F)), ctypes.byref(n))

    assert size() == OK and n.value >= 6 * (64 + 5 * 96)
    need = n.value
    assert L.grouped_mlp_int8_sizes(None, None) == size(E=0) == EINVAL
    assert size(E=129) == size(R=1 << 24) == size(H=131072) == size(F=131072) == EUNSUPPORTED
    assert size(R=-1) == size(H=48) == size(F=0) == size(F=-32) == ESHAPE
    sizes = (ctypes.c_int64 * 4)(1, 0, 2, 3)

    def run(host=sizes, dev=None, x=FAKE, T=3, row=FAKE, p=None, w1=FAKE, s1=FAKE, w2=FAKE, s2=FAKE, y=FAKE, ws=FAKE,
            nb=need, R=6):
        return L.grouped_mlp_fwd_int8(ctypes.byref(mx._Dims(4, R, 64, 96)), host, dev, x, T, row, p, w1, s1, w2, s2, y, ws,
                                      nb, None)

    assert run(host=None) == run(dev=FAKE) == EINVAL
    assert run(x=None) == run(w1=None) == run(s1=None) == run(w2=None) == run(s2=None) == run(y=None) == run(ws=None) == EINVAL
    assert run(R=7) == run(T=-1) == ESHAPE
    assert run(x=ODD) == run(row=ODD) == run(p=ODD) == run(w1=ODD) == run(s1=ODD) == run(w2=ODD) == run(s2=ODD) == EALIGN
    assert run(y=ODD) == run(ws=ctypes.c_void_p(0x100010)) == run(host=None, dev=ODD) == EALIGN
    assert run(nb=need - 1) == EWORKSPACE
    assert run(host=(ctypes.c_int64 * 4)(0, 0, 0, 0), R=0, x=None, nb=0) == OK


def test_binding_refuses_cpu_and_misfitting_tensors(L):
    z, idx = torch.zeros((3, 8)), torch.zeros((3, 2), dtype=torch.int32)
    q, s = torch.zeros((3, 32), dtype=torch.int8), torch.zeros(3)
    for call in (lambda: mx.mx_moe_balance(z, idx), lambda: mx.mx_moe_balance_bwd(z, None, 2),
                 lambda: mx.mx_quantize_int8(torch.zeros((3, 32))), lambda: mx.mx_quantize_int8(torch.zeros(32)),
                 lambda: mx.mx_gemm_int8(q, s, q, s), lambda: mx.mx_grouped_gemm_int8(q, s, q[None], s[None], [3]),
                 lambda: mx.grouped_mlp_fwd_int8(q, None, q, s, q, s, [3])):
        with pytest.raises(ValueError):
            call()
    assert {"mx_moe_balance", "mx_moe_balance_bwd", "MoEBalance", "mx_quantize_int8", "mx_gemm_int8",
            "mx_grouped_gemm_int8", "grouped_mlp_fwd_int8"} <= set(mx.__all__)

"""Refusals of the few-token calls and the router, without a GPU: bad
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


def test_gemv_refusals(L):
    def fp4(x=FAKE, ldx=64, w=FAKE, ws=FAKE, m=2, n=5, k=64, y=FAKE, dt=0, wk=None, nb=0):
        return L.mx_gemv_fp4(x, ldx, w, ws, m, n, k, y, dt, wk, nb, None)

    def nv(x=FAKE, ldx=64, w=FAKE, ws=FAKE, am=FAKE, m=2, n=5, k=64, y=FAKE, dt=1, wk=None, nb=0):
        return L.mx_gemv_nvfp4(x, ldx, w, ws, am, m, n, k, y, dt, wk, nb, None)

    assert fp4(x=None) == fp4(w=None) == fp4(ws=None) == fp4(y=None) == nv(am=None) == EINVAL
    assert fp4(dt=2) == EINVAL
    for k in (0, -32, 16, 48, 33):
        assert fp4(k=k) == nv(k=k) == ESHAPE
    assert fp4(m=-1) == fp4(n=-1) == fp4(ldx=56) == fp4(ldx=68) == fp4(ldx=-64) == ESHAPE
    assert fp4(m=65537) == fp4(n=(1 << 30) + 1) == fp4(k=(1 << 24) + 32, ldx=1 << 25) == EUNSUPPORTED
    assert fp4(ldx=(1 << 24) + 8) == EUNSUPPORTED
    assert fp4(x=ODD) == fp4(w=ODD) == fp4(y=ODD) == nv(ws=ODD) == nv(am=ODD) == EALIGN
    assert b"mx_gemv_nvfp4" in L.mx_last_error()
    assert fp4(m=0) == fp4(n=0) == nv(m=0, x=None) == OK
    # a product that splits k over workgroups needs its planes
    n = ctypes.c_size_t()
    assert L.mx_gemv_sizes(16, 4096, 14336, ctypes.byref(n)) == OK and n.value == 0
    assert L.mx_gemv_sizes(40, 4096, 14336, ctypes.byref(n)) == OK and n.value % (40 * 4096 * 4) == 0 and n.value > 0
    big = dict(m=40, n=4096, k=14336, ldx=14336)
    assert fp4(**big) == nv(**big) == EINVAL
    assert fp4(**big, wk=FAKE, nb=n.value - 1) == nv(**big, wk=FAKE, nb=0) == EWORKSPACE
    assert fp4(**big, wk=ctypes.c_void_p(0x100010), nb=n.value) == EALIGN
    assert L.mx_gemv_sizes(1, 1, 31, None) == L.mx_gemv_sizes(-1, 1, 32, None) == ESHAPE
    assert L.mx_gemv_sizes(65537, 1, 32, None) == EUNSUPPORTED


def test_decode_refusals(L):
    n = ctypes.c_size_t()

    def size(E=4, T=3, H=64, F=96, k=2):
        return L.grouped_mlp_decode_sizes(ctypes.byref(mx._Dims(E, T, H, F)), k, ctypes.byref(n))

    assert size() == OK and n.value >= 3 * 2 * 96 * 4
    need = n.value
    assert size(E=0) == EINVAL and size(E=129) == EUNSUPPORTED
    assert size(H=48) == size(F=48) == size(H=0) == size(F=-32) == size(T=-1) == size(k=0) == ESHAPE
    assert size(T=513) == size(T=2 ** 40) == size(T=1, k=1025) == size(k=2 ** 31 - 1) == EUNSUPPORTED
    assert size(T=1024, k=1) == OK
    assert size(T=1, k=64) == size(T=16, k=64) == OK and size(T=1, k=65) == EUNSUPPORTED
    assert size(H=1 << 19) == size(F=1 << 19) == OK
    assert size(H=(1 << 19) + 32) == size(F=(1 << 19) + 32) == size(F=1 << 62) == EUNSUPPORTED
    assert L.grouped_mlp_decode_sizes(None, 2, ctypes.byref(n)) == EINVAL

    def run(fmt=2, x=FAKE, idx=FAKE, wt=FAKE, w1=FAKE, s1=FAKE, w2=FAKE, s2=FAKE, y=FAKE, ws=FAKE, nb=need, T=3):
        return L.grouped_mlp_decode(ctypes.byref(mx._Dims(4, T, 64, 96)), 2, fmt, x, idx, wt, w1, s1, w2, s2, y, ws,
                                    nb, None)

    assert run(fmt=3) == run(fmt=-1) == EINVAL
    assert run(x=None) == run(idx=None) == run(w1=None) == run(w2=None) == run(y=None) == run(ws=None) == EINVAL
    assert run(s1=None) == run(s2=None) == run(fmt=1, s1=None) == run(fmt=0) == run(fmt=0, s1=None) == EINVAL
    assert run(nb=need - 1) == EWORKSPACE
    assert run(x=ODD) == run(w1=ODD) == run(w2=ODD) == run(y=ODD) == run(idx=ODD) == run(wt=ODD) == EALIGN
    assert run(ws=ctypes.c_void_p(0x100010)) == EALIGN
    assert run(T=0, x=None, nb=0) == OK


def test_route_refusals(L):
    def fwd(z=FAKE, dt=1, T=3, E=8, k=2, idx=FAKE, w=FAKE, lse=FAKE, b=None):
        return L.mx_moe_route(z, dt, b, T, E, k, 1, idx, w, lse, None)

    def bwd(z=FAKE, dt=1, b=None, idx=FAKE, w=FAKE, lse=FAKE, dw=FAKE, rows=6, perm=None, T=3, E=8, k=2, renorm=0, dz=FAKE):
        return L.mx_moe_route_bwd(z, dt, b, idx, w, lse, dw, rows, perm, T, E, k, renorm, dz, None)

    for f in (fwd, bwd):
        assert f(z=None) == f(idx=None) == f(w=None) == f(lse=None) == f(dt=5) == EINVAL
        assert f(T=-1) == f(k=0) == f(k=9) == f(E=0, k=0) == ESHAPE
        assert f(E=129) == EUNSUPPORTED
        assert f(z=ODD) == f(idx=ODD) == f(w=ODD) == f(lse=ODD) == f(b=ODD) == EALIGN
    assert fwd(E=32, k=17) == bwd(E=32, k=17) == fwd(T=(1 << 27) + 1) == EUNSUPPORTED
    assert bwd(rows=5) == bwd(rows=-1, perm=FAKE) == ESHAPE
    assert bwd(dw=None) == bwd(dz=None) == EINVAL
    assert bwd(dw=ODD) == bwd(perm=ODD) == bwd(dz=ODD) == EALIGN
    assert fwd(T=0, z=None) == bwd(T=0, rows=0, z=None) == OK


def test_binding_refuses_what_does_not_fit():
    cpu = torch.zeros((2, 64), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    idx, w = torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2))
    w1, w2 = torch.zeros((3, 64, 64), dtype=torch.bfloat16), torch.zeros((3, 64, 32), dtype=torch.bfloat16)
    if not os.path.exists(mx.lib_path()):
        pytest.skip("library not built")
    for call in (lambda: mx.mx_gemv_fp4(cpu, q, s), lambda: mx.mx_gemv_nvfp4(cpu, q, s, torch.zeros(1)),
                 lambda: mx.mx_gemv_fp4(None, q, s), lambda: mx.grouped_mlp_decode(cpu, idx, w, w1, w2),
                 lambda: mx.mx_moe_route(torch.zeros((2, 8)), 2),
                 lambda: mx.mx_moe_route_bwd(torch.zeros((2, 8)), idx, w, torch.zeros(2), w)):
        with pytest.raises(ValueError):
            call()


def test_what_a_call_allocates_is_memory_of_its_stream(monkeypatch):
    """A call that is given a stream takes its memory from that stream's pool:
    a block freed on the caller's stream may have work queued there that writes
    it still. Results are recorded on the caller's stream, scratch is not."""
    dev = torch.device("cuda", 0)

    class Stream:
        device = dev

    class Tensor:
        def __init__(self, n):
            self.n, self.pool, self.recorded = n, entered[-1], []

        def numel(self):
            return self.n

        def record_stream(self, s):
            self.recorded.append(s)

    class entering:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            entered.append(self.s)

        def __exit__(self, *_):
            entered.pop()

    caller, side = Stream(), Stream()
    entered = [caller]
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Tensor(shape[0]))
    monkeypatch.setattr(torch.cuda, "stream", entering)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: entered[-1])
    out = mx._new((8,), torch.float32, dev, side)
    assert out.pool is side and out.recorded == [caller]
    ws = mx._scratch("a call", None, 512, dev, side)
    assert ws.pool is side and ws.recorded == []
    assert mx._scratch("a call", None, 0, dev, side) is None
    for t in (mx._new((8,), torch.float32, dev, None), mx._scratch("a call", None, 512, dev, None)):
        assert t.pool is caller and t.recorded == []
    assert entered == [caller]


def test_sizes_whose_launch_would_pass_the_thread_limit_are_refused(L):
    """A launch has fewer than 2^32 threads along x: 256 of them take 64 weight
    rows (wide products) or 8 tokens (more than 64 experts)."""
    n = ctypes.c_size_t()
    most = (1 << 30) - 64
    for m in (1, 9, 64):
        assert L.mx_gemv_sizes(m, most, 32, ctypes.byref(n)) == OK
        for over in (most + 1, 1 << 30):
            assert L.mx_gemv_sizes(m, over, 32, ctypes.byref(n)) == EUNSUPPORTED
            assert L.mx_gemv_fp4(FAKE, 32, FAKE, FAKE, m, over, 32, FAKE, 0, None, 0, None) == EUNSUPPORTED
    for over in ((1 << 27) - 7, 1 << 27):
        assert L.mx_moe_route(FAKE, 0, None, over, 128, 2, 1, FAKE, FAKE, FAKE, None) == EUNSUPPORTED
        assert L.mx_moe_route_bwd(FAKE, 0, None, FAKE, FAKE, FAKE, FAKE, over * 2, None, over, 128, 2, 1, FAKE,
                                  None) == EUNSUPPORTED


def test_counts_past_32_bits_are_refused_not_cut(L):
    for E, k in ((4, 2 ** 32 + 2), (2 ** 32 + 4, 2), (4, 2 ** 31)):
        with pytest.raises(mx.MXError):
            mx.mlp_decode_workspace_bytes(E, 3, 64, 96, k)

"""Calls on a stream of the caller's choice: what a call allocates is memory of
the stream that writes it. A block that was just freed on the caller's stream
may have work queued there that writes it still."""
import ast
import inspect

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_mx_amd as mx


def _functions():
    return [f for f in ast.walk(ast.parse(inspect.getsource(mx))) if isinstance(f, ast.FunctionDef)
            and any(a.arg == "stream" for a in f.args.args + f.args.kwonlyargs)]


def test_every_allocation_of_a_call_names_its_stream():
    """In every function that takes a stream: no torch.empty of its own (but in
    the allocators), and the stream handed on to all that allocate."""
    seen = 0
    for f in _functions():
        for c in ast.walk(f):
            if not isinstance(c, ast.Call):
                continue
            name = ast.unparse(c.func)
            assert name not in ("torch.empty", "torch.zeros") or f.name in ("_alloc", "_new"), (f.name, ast.unparse(c))
            if name in ("_alloc", "_new", "_byte_buffer", "_scratch", "WeightCache"):
                passed = [ast.unparse(a) for a in c.args] + [ast.unparse(k.value) for k in c.keywords]
                assert "stream" in passed, (f.name, ast.unparse(c))
                seen += 1
    assert seen > 60


def test_the_streams_device_is_checked():
    class Stream:
        device = torch.device("cuda", 1)

    for dev in ("cuda", "cuda:1", torch.device("cuda"), torch.device("cuda", 1)):
        mx._on_device(Stream(), dev)
    for dev in ("cuda:0", torch.device("cuda", 0), "cpu", torch.device("cpu")):
        with pytest.raises(ValueError):
            mx._on_device(Stream(), dev)


@pytest.mark.gpu
def test_weight_cache_of_a_stream(gpu_lib):
    side = torch.cuda.Stream()
    cache = gpu_lib.WeightCache(2, 128, 128, stream=side)
    assert cache.buf.device == side.device and cache.buf.numel() == gpu_lib.grouped_mlp_weight_cache_bytes(2, 128, 128)


@pytest.mark.gpu
def test_streams_that_do_not_wait_for_the_callers(gpu_lib):
    """Blocks of the sizes that the calls allocate were just freed on the
    caller's stream, whose work on them is still queued when the calls run on
    another stream; the results are those of the caller's stream."""
    gen = torch.Generator().manual_seed(40)
    E, H, F, T, k = 4, 256, 256, 512, 2
    sizes = [256, 0, 100, 156]
    R = sum(sizes)

    def bf16(*shape):
        return (0.1 * torch.randn(shape, generator=gen)).to(torch.bfloat16).cuda()

    x, w1, w2, dy = bf16(R, H), bf16(E, 2 * F, H), bf16(E, H, F), bf16(R, H)
    probs = torch.rand(R, generator=gen).cuda()
    idx = torch.from_numpy(np.random.default_rng(1).integers(0, E, size=(T, k)).astype(np.int32)).cuda()
    idx[:, 1] = (idx[:, 0] + 1) % E
    wt = torch.rand((T, k), generator=gen).cuda()
    cache, cache4 = gpu_lib.grouped_mlp_quantize_weights(w1, w2), gpu_lib.grouped_mlp_fp4_quantize_weights(w1, w2)
    q8 = gpu_lib.quantize(x, colwise=False)
    wq8 = gpu_lib.quantize(w1.view(-1, H), colwise=False)
    q4, s4 = gpu_lib.mx_quantize_fp4(x)
    wq4, ws4 = gpu_lib.mx_quantize_fp4(w1[0])
    perm = gpu_lib.mx_moe_dispatch(x[:T], idx, wt, E)[2]
    rows = bf16(T * k, H)
    states = [gpu_lib.grouped_mlp_fwd(x, probs, w1, w2, sizes)[1], gpu_lib.grouped_mlp_fwd_fp4(x, probs, w1, w2, sizes)[1]]
    calls = [lambda st: list(gpu_lib.quantize(x, stream=st).values()),
             lambda st: [gpu_lib.grouped_gemm(gpu_lib.MX_GROUP_M, sizes, q8["q_row"], q8["s_row"], wq8["q_row"],
                                              wq8["s_row"], N=2 * F, K=H, b_group_stride=2 * F * H, stream=st)],
             lambda st: [gpu_lib.grouped_mlp_fwd(x, probs, w1, w2, sizes, stream=st)[0]],
             lambda st: gpu_lib.grouped_mlp_bwd(dy, probs, states[0], stream=st),
             lambda st: [gpu_lib.grouped_mlp_fwd_cached(x, probs, cache, sizes, stream=st)[0]],
             lambda st: [gpu_lib.grouped_mlp_fwd_cached(x, probs, gpu_lib.grouped_mlp_quantize_weights(w1, w2, stream=st),
                                                        sizes, stream=st)[0]],
             lambda st: [gpu_lib.grouped_mlp_fwd_fp4(x, probs, w1, w2, sizes, stream=st)[0]],
             lambda st: gpu_lib.grouped_mlp_bwd_fp4(dy, probs, states[1], stream=st),
             lambda st: [gpu_lib.grouped_mlp_fwd_fp4_cached(x, probs, cache4, sizes, stream=st)[0]],
             lambda st: gpu_lib.mx_quantize_fp4(x, colwise=True, stream=st),
             lambda st: [gpu_lib.mx_gemm_fp4(q4, s4, wq4, ws4, stream=st)],
             lambda st: gpu_lib.mx_quantize_nvfp4(x, stream=st),
             lambda st: gpu_lib.mx_moe_dispatch(x[:T], idx, wt, E, stream=st),
             lambda st: [gpu_lib.mx_moe_combine(rows, perm, stream=st)]]
    wants = [[t for t in c(None) if t is not None] for c in calls]
    fws, sv, bws = gpu_lib.mlp_sizes(E, R, H, F, sizes)
    blocks = {t.numel() * t.element_size() for w in wants for t in w} | {fws, sv, bws}
    busy = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(20):
            busy = torch.mm(busy, busy).clamp_(-1, 1)
        held = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sorted(blocks) for _ in range(3)]
        del held                                                     # free, and not yet written
        got = [[t for t in c(side) if t is not None] for c in calls]
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, wants)):
            assert len(a) == len(b)
            for u, v in zip(a, b):
                assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)), i

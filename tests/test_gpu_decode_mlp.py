"""The MoE MLP of a few tokens (grouped_mlp_decode) against the 64-bit form
with derived elementwise bounds, for bf16, MXFP8 and MXFP4 weights, and the
whole serving path: router's choice, then the few-token MLP ("Efficient MoE
training for biological foundation models", Key technical approaches item 3)."""
import numpy as np
import pytest
import torch

from tests import decode_ref as ref
from tests.gpu_util import canaries_intact, guarded

pytestmark = pytest.mark.gpu


def _weights(mx, E, H, F, fmt, gen):
    """(arguments of the call, w1 and w2 in float64)."""
    w1 = (0.05 * torch.randn((E, 2 * F, H), generator=gen)).to(torch.bfloat16).cuda()
    w2 = (0.05 * torch.randn((E, H, F), generator=gen)).to(torch.bfloat16).cuda()
    if fmt == "bf16":
        return (w1, w2, None, None), ref.f64(w1), ref.f64(w2)
    out = []
    for w in (w1, w2):
        flat = w.view(-1, w.shape[-1])
        if fmt == "mxfp8":
            d = mx.quantize(flat, colwise=False)
            q, s = d["q_row"], d["s_row"]
        else:
            q, s = mx.mx_quantize_fp4(flat)
        val = ref.mxfp8 if fmt == "mxfp8" else ref.mxfp4
        out.append((q.view(*w.shape[:2], -1), s.view(*w.shape[:2], -1),
                    val(q.cpu().numpy(), s.cpu().numpy()).reshape(w.shape)))
    return (out[0][0], out[1][0], out[0][1], out[1][1]), out[0][2], out[1][2]


def _choices(rng, T, k, E):
    return np.array([rng.permutation(E)[:k] for _ in range(T)], dtype=np.int32).reshape(T, k)


def _check(mx, x, idx, wt, args, w1, w2, out=None):
    y = mx.grouped_mlp_decode(x, torch.from_numpy(idx).cuda(), None if wt is None else torch.from_numpy(wt).cuda(),
                              *args, out=out)
    want, bound = ref.moe(ref.f64(x), idx, np.ones(idx.shape) if wt is None else wt.astype(np.float64), w1, w2)
    err = np.abs(ref.f64(y) - want)
    assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-300)))
    return y


CASES = [(1, 1, 1, 32, 32), (1, 2, 4, 64, 96), (3, 2, 4, 256, 512), (5, 2, 3, 160, 288), (8, 1, 2, 96, 64),
         (9, 3, 5, 128, 160), (16, 2, 2, 64, 544), (17, 2, 8, 96, 128), (33, 1, 1, 64, 96), (40, 4, 4, 32, 32),
         (64, 2, 8, 160, 96), (65, 2, 3, 64, 64), (100, 3, 4, 64, 32), (13, 6, 64, 64, 64), (4, 8, 128, 32, 32),
         (128, 8, 128, 32, 64), (1, 64, 128, 64, 32)]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("T,k,E,H,F", CASES)
def test_against_the_definition(gpu_lib, fmt, T, k, E, H, F):
    gen = torch.Generator().manual_seed(T * 100 + k + E + H + F)
    rng = np.random.default_rng(T + E)
    args, w1, w2 = _weights(gpu_lib, E, H, F, fmt, gen)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    idx = _choices(rng, T, k, E)
    wt = rng.uniform(0, 1, size=(T, k)).astype(np.float32)
    buf, out = guarded((T, H), torch.bfloat16)
    y = _check(gpu_lib, x, idx, wt, args, w1, w2, out=out)
    assert canaries_intact(buf)
    again = gpu_lib.grouped_mlp_decode(x, torch.from_numpy(idx).cuda(), torch.from_numpy(wt).cuda(), *args)
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))


# rows a multiple of 4096 bytes apart; many splits of a long ffn dimension; a
# hidden dimension of a few tiles; the longest sums of planes
WIDE = [("bf16", 20, 2, 3, 2048, 96), ("bf16", 20, 2, 3, 96, 2048), ("mxfp8", 33, 1, 2, 4096, 64),
        ("mxfp8", 18, 2, 4, 64, 4096), ("mxfp4", 24, 3, 4, 8192, 32), ("mxfp4", 64, 2, 2, 32, 8192),
        ("bf16", 8, 4, 8, 64, 2080), ("mxfp4", 1, 2, 9, 96, 8224), ("mxfp8", 20, 1, 1, 64, 8736),
        ("mxfp4", 16, 8, 128, 160, 1056), ("mxfp8", 16, 8, 40, 2080, 96), ("mxfp4", 30, 34, 60, 32, 512)]


@pytest.mark.parametrize("fmt,T,k,E,H,F", WIDE)
def test_long_and_paged_rows(gpu_lib, fmt, T, k, E, H, F):
    gen = torch.Generator().manual_seed(T + k + E + H + F)
    rng = np.random.default_rng(T + E)
    args, w1, w2 = _weights(gpu_lib, E, H, F, fmt, gen)
    x = (0.25 * torch.randn((T, H), generator=gen)).to(torch.bfloat16).cuda()
    idx = _choices(rng, T, k, E)
    idx[rng.uniform(size=idx.shape) < 0.1] = -1
    _check(gpu_lib, x, idx, rng.uniform(0, 1, size=(T, k)).astype(np.float32), args, w1, w2)


def test_two_calls_at_once(gpu_lib):
    """Calls on two streams, each with what it allocates itself, interleaved."""
    gen = torch.Generator().manual_seed(22)
    sizes = [(6, 256, 512, 40, 2), (4, 512, 288, 9, 1)]
    calls, wants = [], []
    for E, H, F, T, k in sizes:
        args, _, _ = _weights(gpu_lib, E, H, F, "mxfp8", gen)
        x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
        idx = torch.from_numpy(_choices(np.random.default_rng(T), T, k, E)).cuda()
        calls.append((x, idx, None, *args))
        wants.append(gpu_lib.grouped_mlp_decode(*calls[-1]))
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    got = [[gpu_lib.grouped_mlp_decode(*c, stream=s) for c, s in zip(calls, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(a, b) for a, b in zip(pair, wants))


def test_a_stream_of_another_device_is_refused(gpu_lib):
    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 1), 0

    gen = torch.Generator().manual_seed(23)
    args, _, _ = _weights(gpu_lib, 2, 32, 32, "bf16", gen)
    x, idx = torch.zeros((1, 32), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    z = torch.zeros((2, 8), device="cuda")
    for call in (lambda: gpu_lib.grouped_mlp_decode(x, idx, None, *args, stream=Elsewhere()),
                 lambda: gpu_lib.mx_moe_route(z, 2, stream=Elsewhere())):
        with pytest.raises(ValueError):
            call()


def test_workspace_of_a_call_on_another_stream(gpu_lib):
    """The call's own workspace is not handed out again before the stream that
    it was given has run the call."""
    gen = torch.Generator().manual_seed(21)
    E, H, F, T, k = 8, 512, 1024, 64, 2
    args, _, _ = _weights(gpu_lib, E, H, F, "mxfp4", gen)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    idx = torch.from_numpy(_choices(np.random.default_rng(1), T, k, E)).cuda()
    want = gpu_lib.grouped_mlp_decode(x, idx, None, *args)
    out = torch.empty_like(want)
    nbytes = gpu_lib.mlp_decode_workspace_bytes(E, T, H, F, k)
    big = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = torch.mm(big, big).clamp_(-1, 1)
    gpu_lib.grouped_mlp_decode(x, idx, None, *args, out=out, stream=side)
    later = [torch.zeros(nbytes, dtype=torch.uint8, device="cuda") for _ in range(3)]
    side.synchronize()
    assert torch.equal(out, want) and all(not t.any() for t in later)


@pytest.mark.parametrize("T", [2, 37])
def test_dropped_repeated_and_unweighted_choices(gpu_lib, T):
    gen = torch.Generator().manual_seed(5)
    rng = np.random.default_rng(6)
    E, H, F, k = 5, 64, 96, 4
    args, w1, w2 = _weights(gpu_lib, E, H, F, "mxfp4", gen)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    idx = rng.integers(0, E, size=(T, k)).astype(np.int32)           # an expert may come twice
    idx[0] = [-1, E, 2 ** 31 - 1, -2 ** 31]                          # nothing left of this token
    idx[1, 2] = -1
    y = _check(gpu_lib, x, idx, None, args, w1, w2)
    assert not y[0].any()
    y = _check(gpu_lib, x, idx, rng.uniform(-1, 1, size=(T, k)).astype(np.float32), args, w1, w2)
    assert not y[0].any()
    none = gpu_lib.grouped_mlp_decode(x, torch.full((T, k), -1, dtype=torch.int32, device="cuda"), None, *args)
    assert not none.any()
    assert gpu_lib.grouped_mlp_decode(x[:0], torch.empty((0, k), dtype=torch.int32, device="cuda"), None, *args).shape == (0, H)


def test_every_token_on_one_expert_and_unread_experts(gpu_lib):
    """Experts that no token names may hold anything (here NaN codes)."""
    gen = torch.Generator().manual_seed(8)
    E, H, F, T = 4, 96, 64, 50
    args, w1, w2 = _weights(gpu_lib, E, H, F, "mxfp8", gen)
    for a in args[:2]:
        a[[0, 1, 3]] = 0x7F
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    idx = np.full((T, 1), 2, dtype=np.int32)
    _check(gpu_lib, x, idx, None, args, np.nan_to_num(w1), np.nan_to_num(w2))


def test_nonfinite_tokens_stay_apart(gpu_lib):
    gen = torch.Generator().manual_seed(10)
    rng = np.random.default_rng(11)
    E, H, F, T, k = 3, 64, 64, 20, 2
    args, _, _ = _weights(gpu_lib, E, H, F, "mxfp4", gen)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    idx = torch.from_numpy(_choices(rng, T, k, E)).cuda()
    clean = gpu_lib.grouped_mlp_decode(x, idx, None, *args)
    x[4, 7], x[9, 0] = float("nan"), float("inf")
    got = gpu_lib.grouped_mlp_decode(x, idx, None, *args)
    keep = [t for t in range(T) if t not in (4, 9)]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[4]).all()


def test_weights_past_four_gib(gpu_lib):
    """The last of 128 experts lies past 2^32 bytes in w1 and past 2^31 elements."""
    E, H, F = 128, 4096, 2304
    w1 = torch.zeros((E, 2 * F, H), dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros((E, H, F), dtype=torch.bfloat16, device="cuda")
    assert w1.numel() * 2 > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(2)
    w1[-1] = (0.05 * torch.randn((2 * F, H), generator=gen, device="cuda")).to(torch.bfloat16)
    w2[-1] = (0.05 * torch.randn((H, F), generator=gen, device="cuda")).to(torch.bfloat16)
    x = torch.randn((2, H), generator=gen, device="cuda").to(torch.bfloat16)
    idx = torch.tensor([[127, 3], [5, 127]], dtype=torch.int32, device="cuda")
    y = gpu_lib.grouped_mlp_decode(x, idx, None, w1, w2)
    want, bound = ref.moe(ref.f64(x), np.zeros((2, 1), dtype=np.int32), np.ones((2, 1)), ref.f64(w1[-1:]), ref.f64(w2[-1:]))
    assert np.all(np.abs(ref.f64(y) - want) <= bound)


def test_on_a_stream_and_in_two_graphs_of_one_workspace(gpu_lib):
    """Two captured calls share a workspace (run one after the other), with
    new tokens and choices at every replay and eager work in between."""
    gen = torch.Generator().manual_seed(12)
    rng = np.random.default_rng(13)
    E, H, F, T, k = 6, 128, 160, 12, 2
    args, _, _ = _weights(gpu_lib, E, H, F, "mxfp4", gen)
    ws = torch.empty(gpu_lib.mlp_decode_workspace_bytes(E, T, H, F, k), dtype=torch.uint8, device="cuda")
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    idx = torch.from_numpy(_choices(rng, T, k, E)).cuda()
    outs, graphs = [torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2)], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = gpu_lib.grouped_mlp_decode(x, idx, None, *args)
    gpu_lib.grouped_mlp_decode(x, idx, None, *args, out=outs[0], stream=side)
    side.synchronize()
    assert torch.equal(outs[0], want)
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gpu_lib.grouped_mlp_decode(x, idx, None, *args, out=o, workspace=ws)
        graphs.append(g)
    for i in range(4):
        x.copy_(torch.randn((T, H), generator=gen))
        idx.copy_(torch.from_numpy(_choices(rng, T, k, E)))
        eager = gpu_lib.grouped_mlp_decode(x, idx, None, *args)
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, eager), i


def test_route_then_decode(gpu_lib):
    """Serving: logits -> choices and weights -> MLP, against the same in 64 bits."""
    gen = torch.Generator().manual_seed(20)
    E, H, F, T, k = 8, 128, 96, 11, 2
    args, w1, w2 = _weights(gpu_lib, E, H, F, "mxfp4", gen)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    logits = torch.randn((T, E), generator=gen).to(torch.bfloat16).cuda()
    logits[3, 1:] = float("-inf")                                    # one expert open: the second choice is dropped
    logits[6] = float("-inf")                                        # none
    idx, w, _ = gpu_lib.mx_moe_route(logits, k)
    y = gpu_lib.grouped_mlp_decode(x, idx, w, *args)
    ridx, rw, _, rel, _ = ref.route(ref.f64(logits), None, k, True)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    want, bound = ref.moe(ref.f64(x), ridx, rw, w1, w2)
    # a weight that is off by rel moves its part of y by as much: |y| parts sum to what moe's terms bound
    parts = sum(np.abs(ref.moe(ref.f64(x), ridx[:, j:j + 1], rw[:, j:j + 1], w1, w2)[0]) for j in range(k))
    assert np.all(np.abs(ref.f64(y) - want) <= bound + 2 * rel * parts)
    assert not y[6].any()


@pytest.mark.parametrize("T", [4, 64])
def test_a_stream_that_does_not_wait_for_the_callers(gpu_lib, T):
    """Blocks of the sizes that the call allocates were just freed on the
    caller's stream, whose work on them is still queued when the call runs on
    another stream: neither side writes the other's memory."""
    gen = torch.Generator().manual_seed(24)
    E, H, F, k = 8, 512, 1024, 2
    args, _, _ = _weights(gpu_lib, E, H, F, "mxfp4", gen)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).cuda()
    z = torch.randn((T, E), generator=gen).cuda()
    idx, w, lse = gpu_lib.mx_moe_route(z, k)
    q, s = args[0][0], args[2][0]                                    # one expert's first matrix, [2F, H]
    calls = [lambda st: gpu_lib.grouped_mlp_decode(x, idx, w, *args, stream=st),
             lambda st: gpu_lib.mx_gemv_fp4(x, q, s, out_dtype=torch.float32, stream=st),
             lambda st: gpu_lib.mx_moe_route_bwd(z, idx, w, lse, w, stream=st),
             lambda st: gpu_lib.mx_moe_route(z, k, stream=st)]
    sizes = [gpu_lib.mlp_decode_workspace_bytes(E, T, H, F, k), gpu_lib.gemv_workspace_bytes(T, 2 * F, H), T * H * 2,
             T * 2 * F * 4, T * k * 4, T * E * 4, T * 4]
    wants = [c(None) for c in calls]
    busy = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(20):
            busy = torch.mm(busy, busy).clamp_(-1, 1)
        held = [torch.full((max(n, 1),), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        del held                                                     # free, and not yet written
        got = [c(side) for c in calls]
        torch.cuda.synchronize()
        for a, b in zip([*got[:3], *got[3]], [*wants[:3], *wants[3]]):
            assert torch.equal(a, b)


def test_results_freed_while_the_callers_stream_reads_them(gpu_lib):
    """A result that is dropped while the caller's stream has yet to read it is
    not handed to the stream that made it before that read."""
    gen = torch.Generator().manual_seed(25)
    T, E, k = 4096, 64, 8
    z = [torch.randn((T, E), generator=gen).cuda() for _ in range(2)]
    want = gpu_lib.mx_moe_route(z[0], k)[1].sum(1)
    busy = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    idx, w, lse = gpu_lib.mx_moe_route(z[0], k, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(20):
        busy = torch.mm(busy, busy).clamp_(-1, 1)
    got = w.sum(1)                                                   # queued behind the products
    del idx, w, lse
    later = [gpu_lib.mx_moe_route(z[1], k, stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(later) == 3


# All E8M0 scale codes, each with 8 groups of 32 E4M3 codes. NaN codes and values
# from 2^128 on are left out (they would spread over their row): zero instead.
def _all_mxfp8():
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(8, 32), (255, 1))          # [255 * 8, 32]
    scales = np.repeat(np.arange(255, dtype=np.uint8), 8)[:, None]
    with np.errstate(invalid="ignore"):
        codes[~(np.abs(ref.mxfp8(codes, scales)) < 2.0 ** 128)] = 0
    assert (codes[24:247 * 8] == 0).sum() == (247 - 3) * (1 + 2)                      # codes 3 .. 246: zero and the two NaNs
    return codes, scales, ref.mxfp8(codes, scales)


def _check_expanded(got, want):
    """Exact where bf16 has the value: any multiple of 2^-133, its last step
    (under scale codes from 3 on every one is); within that step otherwise."""
    exact = np.ldexp(want, 133) % 1.0 == 0
    assert exact[24:].all() and not exact[:24].all()
    assert np.array_equal(got[exact], want[exact])
    assert np.all(np.abs(got - want) < 2.0 ** -133)


def test_every_mxfp8_code_and_scale_in_the_second_product(gpu_lib):
    """Tokens and experts that make A a unit matrix pick single weights: token t
    has g = 32 and u = 1 at f = t only, and weight 2^-5 (silu(32) is 32 in fp32,
    silu(0) is 0)."""
    codes, scales, want = _all_mxfp8()
    H, F = 2048, 32
    w2, s2 = np.zeros((1, H, F), dtype=np.uint8), np.full((1, H, 1), 127, dtype=np.uint8)
    w2[0, :2040], s2[0, :2040] = codes, scales
    w1 = np.zeros((1, 2 * F, H), dtype=np.uint8)
    w1[0, np.arange(F), np.arange(F)], w1[0, F + np.arange(F), np.arange(F)] = 0x60, 0x38       # 32 and 1
    s1 = np.full((1, 2 * F, H // 32), 127, dtype=np.uint8)
    put = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    x = torch.eye(F, H).to(torch.bfloat16).cuda()
    idx, wt = torch.zeros((F, 1), dtype=torch.int32, device="cuda"), torch.full((F, 1), 2.0 ** -5, device="cuda")
    for T in (4, 16, 32):
        y = gpu_lib.grouped_mlp_decode(x[:T], idx[:T], wt[:T], put(w1), put(w2), put(s1), put(s2))
        if T == 32:
            _check_expanded(ref.f64(y).T[:2040], want)
        else:
            full = gpu_lib.grouped_mlp_decode(x, idx, wt, put(w1), put(w2), put(s1), put(s2))
            assert torch.equal(y, full[:T])


def test_every_mxfp8_code_and_scale_in_the_first_product(gpu_lib):
    """The codes as rows of u, g = 32 everywhere, W2 a unit matrix: y[t, f] is
    expert t / 32's weight f under the unit token t % 32."""
    codes, scales, want = _all_mxfp8()
    H = F = 32
    put = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    E = 32
    x = torch.eye(H).repeat(E, 1).to(torch.bfloat16).cuda()
    idx = torch.arange(E, dtype=torch.int32).repeat_interleave(H)[:, None].contiguous().cuda()
    wt = torch.full((E * H, 1), 2.0 ** -5, device="cuda")
    w2, s2 = np.tile((np.eye(H) * 0x38).astype(np.uint8), (E, 1, 1)), np.full((E, H, 1), 127, dtype=np.uint8)
    got = np.zeros_like(want)
    for r0 in (0, 2040 - E * F):
        w1 = np.full((E, 2 * F, H), 0x60, dtype=np.uint8)
        s1 = np.full((E, 2 * F, 1), 127, dtype=np.uint8)
        w1[:, F:], s1[:, F:] = codes[r0:r0 + E * F].reshape(E, F, H), scales[r0:r0 + E * F].reshape(E, F, 1)
        y = ref.f64(gpu_lib.grouped_mlp_decode(x, idx, wt, put(w1), put(w2), put(s1), put(s2)))
        got[r0:r0 + E * F] = y.reshape(E, H, F).transpose(0, 2, 1).reshape(E * F, H)
    _check_expanded(got, want)


def test_weights_that_the_cast_makes_of_bf16_are_exact(gpu_lib):
    """bf16 weights down to its last subnormal, cast to MXFP8: every value that
    the cast makes is a multiple of 2^-133 below 2^128."""
    rng = np.random.default_rng(26)
    bits = rng.integers(0, 2 ** 16, size=(512, 256)).astype(np.uint16)
    bits[:256] &= 0x81FF                                             # magnitudes below 2^-123
    bits[256:384] = (bits[256:384] & 0x80FF) | 0x7E00                # magnitudes from 2^125 on
    bits[(bits & 0x7F80) == 0x7F80] = 0                              # no infinities, no NaN
    d = gpu_lib.quantize(torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16), colwise=False)
    v = ref.mxfp8(d["q_row"].cpu().numpy(), d["s_row"].cpu().numpy())
    assert np.all(np.abs(v) < 2.0 ** 128) and np.all(np.ldexp(v, 133) % 1.0 == 0)

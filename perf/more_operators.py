"""Workloads of the router's balance loss (mx_moe_balance and its backward) and of
the experts in 8-bit integers: the cast with one scale per row (mx_quantize_int8),
the product with scales for each token and channel (mx_gemm_int8,
mx_grouped_gemm_int8) and the MoE MLP on such weights (grouped_mlp_fwd_int8).

Shapes: hidden 4096, ffn 14336, 8 experts top-2 and the tiny MoE case (256, 512,
4 experts) are those of this repository's workloads; the others are generic.
Weights are normal draws, cast here in torch; activations have a few channels
that are much larger than the rest.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # balance of a small micro-batch over many experts: latency
        {"name": "balance T33 e128", "op": "balance", "tokens": 33, "experts": 128, "topk": 8, "dtype": "bf16", "segs": 0,
         "bias": True},
        # a training step's packed sequences with padding behind the last, a loss for each sequence
        {"name": "balance T16383 e128 s13", "op": "balance", "tokens": 16383, "experts": 128, "topk": 8, "dtype": "bf16",
         "segs": 13, "bias": False},
        # gradient of one loss over a training step's tokens
        {"name": "balance bwd T8192 e8", "op": "balance_bwd", "tokens": 8192, "experts": 8, "topk": 2, "dtype": "f32", "segs": 0,
         "bias": False, "add": False, "dprob": False},
        # gradients of the losses and of the mean probabilities, added to the router's own gradient
        {"name": "balance bwd T16383 e128 s13", "op": "balance_bwd", "tokens": 16383, "experts": 128, "topk": 8,
         "dtype": "bf16", "segs": 13, "bias": True, "add": True, "dprob": True},
        # cast of a decoding batch's activations
        {"name": "cast8 33x4096", "op": "cast", "rows": 33, "from": 33, "cols": 4096, "dtype": "bf16", "index": False,
         "weight": False},
        # cast of a training step's routed rows, read through the dispatch's index, routing weights in the scales
        {"name": "cast8 gather 16384x4096", "op": "cast", "rows": 16384, "from": 8192, "cols": 4096, "dtype": "bf16",
         "index": True, "weight": True},
        # one row against a small projection of odd size: launch latency
        {"name": "gemm8 1x999 k544", "op": "gemm", "m": 1, "n": 999, "k": 544, "groups": 0, "out": "bf16"},
        # a decoding batch's gate and up projection
        {"name": "gemm8 16x28672 k4096", "op": "gemm", "m": 16, "n": 28672, "k": 4096, "groups": 0, "out": "bf16"},
        # the dense MLP's down projection of a ragged prompt, fp32 results (partial sums of a sharded layer)
        {"name": "gemm8 8191x4096 k14336", "op": "gemm", "m": 8191, "n": 4096, "k": 14336, "groups": 0, "out": "f32"},
        # the experts' gate and up products of a training step's routed rows, row counts on the device
        {"name": "gemm8 e8 8192x28672 k4096", "op": "gemm", "m": 8192, "n": 28672, "k": 4096, "groups": 8, "out": "bf16",
         "counts": "device"},
        # the tiny MoE layer, three tokens: latency of the whole MLP
        {"name": "mlp8 tiny T3", "op": "mlp", "tokens": 3, "topk": 2, "experts": 4, "hidden": 256, "ffn": 512,
         "counts": "device"},
        # a prompt of 4096 tokens through 8 experts
        {"name": "mlp8 T4096 e8", "op": "mlp", "tokens": 4096, "topk": 2, "experts": 8, "hidden": 4096, "ffn": 14336,
         "counts": "host"},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["balance", "balance_bwd", "cast", "gemm", "gemm", "mlp", "mlp"])
    if op in ("balance", "balance_bwd"):
        experts = rng.choice([4, 8, 16, 60, 64, 128])
        case = {"op": op, "tokens": _spread(rng, 1, 16384), "experts": experts, "topk": rng.randint(1, min(8, experts)),
                "dtype": rng.choice(["bf16", "f32"]), "segs": rng.choice([0, 0, 1, 7, 64]), "bias": rng.random() < 0.5}
        if op == "balance_bwd":
            case |= {"add": rng.random() < 0.5, "dprob": rng.random() < 0.5}
        return case
    if op == "cast":
        index = rng.random() < 0.5
        rows = _spread(rng, 1, 16384)
        return {"op": op, "rows": rows, "from": max(1, rows // rng.randint(1, 4)) if index else rows,
                "cols": 16 * _spread(rng, 1, 512), "dtype": rng.choice(["bf16", "f32"]), "index": index,
                "weight": rng.random() < 0.5}
    if op == "gemm":
        groups = rng.choice([0, 0, 4, 8, 60])
        m, n, k = _spread(rng, 1, 8192), _spread(rng, 16, 28672), 16 * _spread(rng, 1, 896)
        while m * n * k > 8192 * 28672 * 4096 or max(1, groups) * n * k > 1e9:
            n = max(16, n // 2)
        return {"op": op, "m": m, "n": n, "k": k, "groups": groups, "out": rng.choice(["bf16", "f32"]),
                "counts": rng.choice(["host", "device"])}
    experts = rng.choice([1, 4, 8, 16, 60])
    topk = rng.randint(1, min(8, experts))
    hidden, ffn = 32 * _spread(rng, 4, 128), 32 * _spread(rng, 4, 448)
    while experts * hidden * ffn > 4.7e8:
        ffn = max(32, ffn // 64 * 32)
    return {"op": op, "tokens": _spread(rng, 1, 8192 // topk), "topk": topk, "experts": experts, "hidden": hidden,
            "ffn": ffn, "counts": rng.choice(["host", "device"])}


# ---- inputs

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _activations(gen, rows, cols):
    """Normal values, one channel in 64 ten times the others."""
    big = 1 + 9 * (torch.rand(cols, generator=gen, device=DEV) < 1 / 64)
    return torch.randn((rows, cols), generator=gen, device=DEV) * big


def _codes(gen, rows, cols, make):
    """A matrix in 8-bit integers with a scale per row, made in pieces of at most 2^27 values."""
    q = torch.empty((rows, cols), dtype=torch.int8, device=DEV)
    s = torch.empty(rows, device=DEV)
    step = max(1, 2 ** 27 // cols)
    for r in range(0, rows, step):
        q[r:r + step], s[r:r + step] = _cast_plain(make(gen, min(step, rows - r), cols))
    return q, s


def _weights(gen, rows, cols):
    return _codes(gen, rows, cols, lambda g, r, c: 0.02 * torch.randn((r, c), generator=g, device=DEV))


def _router_logits(gen, tokens, experts, dtype):
    """Logits of skewed load: a spread per token and one per expert."""
    z = torch.randn((tokens, experts), generator=gen, device=DEV) + 0.7 * torch.randn(experts, generator=gen, device=DEV)
    return z.to(_dtype(dtype))


def _choices(z, bias, k):
    """The k largest keys of a row, from the largest; -1 where fewer experts are open."""
    key = z.float() if bias is None else z.float() + bias
    top, idx = torch.sort(torch.where(key > -math.inf, key, -math.inf), dim=1, descending=True, stable=True)
    return torch.where(top > -math.inf, idx, -1)[:, :k].to(torch.int32).contiguous()


def _segments(gen, tokens, segs):
    """Offsets of ragged sequences (equal cuts make empty ones), with some padding behind the last."""
    if not segs:
        return None
    cuts = torch.randint(0, tokens + 1, (segs,), generator=gen, device=DEV)
    cuts[-1] = tokens - tokens // 50
    return torch.cat([cuts.new_zeros(1), cuts.clamp(max=tokens - tokens // 50).sort()[0]]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("balance", "balance_bwd"):
        t, e = case["tokens"], case["experts"]
        z = _router_logits(gen, t, e, case["dtype"])
        z[torch.rand((t, e), generator=gen, device=DEV) < 0.01] = -math.inf      # a few experts closed to a few tokens
        s["logits"] = z
        s["b"] = 0.1 * torch.randn(e, generator=gen, device=DEV) if case["bias"] else None
        s["topk_idx"] = _choices(z, s["b"], case["topk"])
        s["segments"] = _segments(gen, t, case["segs"])
        if op == "balance_bwd":
            n = max(1, case["segs"])
            s["counts_in"] = _balance_plain(s)["counts"]
            s["dloss"] = 0.01 / n * (1 + torch.rand(n, generator=gen, device=DEV))
            s["dp"] = 1e-2 * torch.randn((n, e), generator=gen, device=DEV) if case["dprob"] else None
            s["base"] = (1e-5 * torch.randn((t, e), generator=gen, device=DEV)).to(z.dtype) if case["add"] else None
    elif op == "cast":
        s["x"] = _activations(gen, case["from"], case["cols"]).to(_dtype(case["dtype"]))
        index = torch.randint(0, case["from"], (case["rows"],), generator=gen, device=DEV).to(torch.int32)
        s["row_index"] = index if case["index"] else None
        s["row_weight"] = torch.rand(case["rows"], generator=gen, device=DEV) if case["weight"] else None
    elif op == "gemm":
        g = case["groups"]
        s["a"] = _codes(gen, case["m"], case["k"], _activations)
        b, bs = _weights(gen, max(1, g) * case["n"], case["k"])
        s["b"] = (b.view(g, case["n"], -1), bs.view(g, -1)) if g else (b, bs)
        if g:
            share = torch.rand(g, generator=gen, device=DEV) + 0.2
            group = torch.multinomial(share, case["m"], replacement=True, generator=gen)
            _counts(s, torch.bincount(group, minlength=g))
    else:
        t, k, e, h, f = case["tokens"], case["topk"], case["experts"], case["hidden"], case["ffn"]
        s["x"] = _activations(gen, t, h).to(torch.bfloat16)
        w1, w1_s = _weights(gen, e * 2 * f, h)
        w2, w2_s = _weights(gen, e * h, f)
        s["w"] = (w1.view(e, 2 * f, h), w1_s.view(e, 2 * f), w2.view(e, h, f), w2_s.view(e, h))
        z = _router_logits(gen, t, e, "f32")
        idx = _choices(z, None, k).long()
        order = torch.argsort(idx.reshape(-1), stable=True)                  # routed rows by expert, then token
        s["row_token"] = (order // k).to(torch.int32)
        s["probs"] = torch.softmax(z.gather(1, idx), 1).reshape(-1)[order]
        _counts(s, torch.bincount(idx.reshape(-1), minlength=e))
    return s


def _counts(s, counts):
    """Rows per group as the program holds them, and for the plain form each row's group and place in it."""
    host = counts.tolist()
    s["sizes"] = counts if s["counts"] == "device" else host
    s["most"] = max(1, max(host))
    ends = counts.cumsum(0)
    row = torch.arange(sum(host), device=DEV)
    s["group"] = torch.searchsorted(ends, row, right=True)
    s["place"] = row - (ends - counts)[s["group"]]


# ---- the plain forms

def _cast_plain(x):
    """Codes by the exact quotient 127 x / top (64 bits: values next to a half), one scale per row."""
    top = x.float().abs().amax(1).clamp(min=2.0 ** -100)
    return torch.round(127 * x.double() / top.double()[:, None]).to(torch.int8), top / 127.0


def _sequence(s):
    """Each token's sequence (the number of sequences where it is in none), and the tokens of each."""
    t, o = s["tokens"], s["segments"]
    if o is None:
        return torch.zeros(t, dtype=torch.long, device=DEV), torch.full((1,), t, device=DEV)
    at = torch.arange(t, dtype=torch.int32, device=DEV)
    return torch.searchsorted(o[1:].contiguous(), at, right=True), o.diff().clamp(min=1)


def _sums(s, v):
    """Sums of v [T, E] over each sequence's tokens, in v's type."""
    if s["segments"] is None:
        return v.sum(0, keepdim=True)
    v = v.T.contiguous()
    run = torch.cat([torch.zeros_like(v[:, :1]), v.cumsum(1)], 1)
    return (run[:, s["segments"][1:].long()] - run[:, s["segments"][:-1].long()]).T.contiguous()


def _probs_plain(s):
    z = s["logits"].float()
    key = z if s["b"] is None else z + s["b"]
    z = torch.where(key > -math.inf, z, -math.inf)
    top = z.amax(1, keepdim=True)
    p = torch.where(z > -math.inf, torch.exp(z - top), 0.0)
    return p / p.sum(1, keepdim=True).clamp(min=1e-30)


def _balance_plain(s):
    n, e = _sequence(s)[1], s["experts"]
    counts = _sums(s, (s["topk_idx"].unsqueeze(-1) == torch.arange(e, device=DEV)).sum(1))
    mean = _sums(s, _probs_plain(s).double()) / n[:, None]
    loss = (counts * mean).sum(1) * e / (s["topk"] * n)
    return {"loss": loss.float(), "counts": counts, "mean_prob": mean.float()}


def _balance_bwd_plain(s):
    seg, n = _sequence(s)
    a = s["counts_in"] * (s["dloss"].double() * s["experts"] / (s["topk"] * n))[:, None]
    if s["dp"] is not None:
        a = a + s["dp"]
    a = torch.cat([a / n[:, None], torch.zeros_like(a[:1])])[seg]            # each token's, 0 outside the sequences
    p = _probs_plain(s)
    dz = (p * (a - (p * a).sum(1, keepdim=True))).float()
    if s["base"] is not None:
        dz = dz + s["base"].float()
    return dz.to(s["logits"].dtype)


def _product(a, a_s, b, b_s):
    return (a.float() @ b.float().mT) * a_s.unsqueeze(-1) * b_s.unsqueeze(-2)


def _grouped(s, a, a_s, b, b_s):
    """The rows of each group times its matrix: groups side by side, filled up to the largest one."""
    g = b.shape[0]
    pad = torch.zeros((g, s["most"], a.shape[1]), device=DEV)
    pad_s = torch.zeros((g, s["most"]), device=DEV)
    pad[s["group"], s["place"]] = a.float()
    pad_s[s["group"], s["place"]] = a_s
    return _product(pad, pad_s, b, b_s)[s["group"], s["place"]]


def _run_plain(s):
    op = s["op"]
    if op == "balance":
        return _balance_plain(s)
    if op == "balance_bwd":
        return _balance_bwd_plain(s)
    if op == "cast":
        x = s["x"] if s["row_index"] is None else s["x"][s["row_index"].long()]
        q, scale = _cast_plain(x)
        if s["row_weight"] is not None:
            scale = scale * s["row_weight"]
        return {"values": q * scale[:, None], "scale": scale}
    if op == "gemm":
        product = _grouped(s, *s["a"], *s["b"]) if s["groups"] else _product(*s["a"], *s["b"])
        return product.to(_dtype(s["out"]))
    w1, w1_s, w2, w2_s = s["w"]
    h = _grouped(s, *_cast_plain(s["x"][s["row_token"].long()]), w1, w1_s)
    g, u = h[:, :s["ffn"]], h[:, s["ffn"]:]
    a, a_s = _cast_plain(g * torch.sigmoid(g) * u)
    return _grouped(s, a, a_s * s["probs"], w2, w2_s).to(torch.bfloat16)


def _run_own(s):
    import mxfp8_block_scaled_mx_amd as mx
    op = s["op"]
    if op == "balance":
        loss, counts, mean_prob = mx.mx_moe_balance(s["logits"], s["topk_idx"], bias=s["b"], segments=s["segments"])
        return {"loss": loss, "counts": counts, "mean_prob": mean_prob}
    if op == "balance_bwd":
        return mx.mx_moe_balance_bwd(s["logits"], s["counts_in"], s["topk"], dloss=s["dloss"], dmean_prob=s["dp"],
                                     bias=s["b"], segments=s["segments"], add=s["base"])
    if op == "cast":
        q, scale = mx.mx_quantize_int8(s["x"], row_index=s["row_index"], row_weight=s["row_weight"])
        return {"values": q * scale[:, None], "scale": scale}
    if op == "gemm":
        if s["groups"]:
            return mx.mx_grouped_gemm_int8(*s["a"], *s["b"], s["sizes"], out_dtype=_dtype(s["out"]))
        return mx.mx_gemm_int8(*s["a"], *s["b"], out_dtype=_dtype(s["out"]))
    w1, w1_s, w2, w2_s = s["w"]
    return mx.grouped_mlp_fwd_int8(s["x"], s["probs"], w1, w1_s, w2, w2_s, s["sizes"], row_token=s["row_token"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op in ("balance", "balance_bwd"):
        t, e, n = case["tokens"], case["experts"], max(1, case["segs"])
        size = 2 if case["dtype"] == "bf16" else 4
        if op == "balance":
            return {"bytes": t * e * size + 4 * t * case["topk"] + 12 * n * e, "flops": 5 * t * e}
        return {"bytes": (3 if case["add"] else 2) * t * e * size + 12 * n * e, "flops": 8 * t * e}
    if op == "cast":
        size = 2 if case["dtype"] == "bf16" else 4
        read = min(case["from"], case["rows"])
        return {"bytes": read * case["cols"] * size + case["rows"] * (case["cols"] + 12), "flops": 3 * case["rows"] * case["cols"]}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        g = max(1, min(case["groups"], m))
        return {"bytes": g * n * (k + 4) + m * (k + 4) + size * m * n, "flops": 2 * m * n * k}
    t, k, e, h, f = case["tokens"], case["topk"], case["experts"], case["hidden"], case["ffn"]
    read = e * (1 - (1 - k / e) ** t)                                        # experts that are chosen, at even odds
    return {"bytes": read * (3 * h * f + 8 * f + 4 * h) + 2 * t * h + 8 * t * k + 2 * t * k * h, "flops": 6 * t * k * h * f}


# ---- the definitions in 64 bits

def _cast64(x):
    x = x.double()
    top = x.abs().amax(1, keepdim=True).clamp(min=2.0 ** -100)
    return torch.round(127 * x / top), top / 127


def _softmax64(z, shut):
    z = torch.where(shut, -1e300, z)
    p = torch.where(shut, 0.0, torch.exp(z - z.detach().amax(1, keepdim=True)))
    return p / p.sum(1, keepdim=True).clamp(min=1e-300)


def _spans(s):
    o = [0, s["tokens"]] if s["segments"] is None else s["segments"].tolist()
    return list(zip(o[:-1], o[1:]))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("balance", "balance_bwd"):
        z = s["logits"].double()
        shut = torch.isinf(z)
        e, k = case["experts"], case["topk"]
    if op == "balance":
        p = _softmax64(z, shut)
        loss, counts, mean = [], [], []
        for b, t in _spans(s):
            ids = s["topk_idx"][b:t].reshape(-1)
            c = torch.bincount(ids[ids >= 0], minlength=e)
            m = p[b:t].sum(0) / max(1, t - b)
            loss.append(e * (c.double() / max(1, k * (t - b))).dot(m))
            counts.append(c)
            mean.append(m)
        return {"loss": torch.stack(loss), "counts": torch.stack(counts), "mean_prob": torch.stack(mean)}
    if op == "balance_bwd":
        # by autograd through the definition of the losses
        z = torch.where(shut, 0.0, z).requires_grad_()
        p = _softmax64(z, shut)
        total = 0.0 * z.sum()
        for i, (b, t) in enumerate(_spans(s)):
            if t > b:
                m = p[b:t].mean(0)
                total = total + s["dloss"][i].double() * e / (k * (t - b)) * (s["counts_in"][i].double() * m).sum()
                if s["dp"] is not None:
                    total = total + (s["dp"][i].double() * m).sum()
        total.backward()
        return z.grad if s["base"] is None else z.grad + s["base"].double()
    if op == "cast":
        x = s["x"] if s["row_index"] is None else s["x"].index_select(0, s["row_index"])
        q, scale = _cast64(x)
        if s["row_weight"] is not None:
            scale = scale * s["row_weight"].double()[:, None]
        return {"values": q * scale, "scale": scale[:, 0]}

    def product(a, a_s, b, b_s):
        return (a.double() @ b.double().T) * a_s.double().view(-1, 1) * b_s.double()

    if op == "gemm" and not case["groups"]:
        return product(*s["a"], *s["b"])
    sizes = s["sizes"].tolist() if case["counts"] == "device" else s["sizes"]
    out, at = [], 0
    for i, n in enumerate(sizes):
        rows = slice(at, at + n)
        at += n
        if op == "gemm":
            out.append(product(s["a"][0][rows], s["a"][1][rows], s["b"][0][i], s["b"][1][i]))
            continue
        w1, w1_s, w2, w2_s = (w[i] for w in s["w"])
        if n:
            h = product(*_cast64(s["x"].index_select(0, s["row_token"][rows])), w1, w1_s)
            g, u = h.chunk(2, 1)
            a, a_s = _cast64(u * g / (1 + torch.exp(-g)))
            out.append(product(a, a_s[:, 0] * s["probs"][rows].double(), w2, w2_s))
    return torch.cat(out)

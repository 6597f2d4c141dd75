"""Workloads of the operators around the experts of an MoE layer: the router
(mx_moe_route and its backward), the few-token MoE MLP (grouped_mlp_decode) and
the products of a few rows with 4-bit weights (mx_gemv_fp4, mx_gemv_nvfp4).

Shapes: hidden 4096, ffn 14336, 8 experts top-2 and the tiny MoE case (256, 512,
4 experts) are those of this repository's workloads; the others are generic.
Weights are normal draws cast to their block format here, in torch.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
FORMAT_BYTES = {"bf16": 2.0, "mxfp8": 1.0 + 1 / 32, "mxfp4": 0.5 + 1 / 32, "nvfp4": 0.5 + 1 / 16}


def listed():
    return [
        # one row against a small projection of odd size: launch latency
        {"name": "gemv4 1x999 k544", "op": "gemv", "fmt": "mxfp4", "m": 1, "n": 999, "k": 544, "out": "bf16"},
        # one token's down projection of the dense MLP
        {"name": "gemv4 1x4096 k14336", "op": "gemv", "fmt": "mxfp4", "m": 1, "n": 4096, "k": 14336, "out": "bf16"},
        # a decoding batch's gate and up projection
        {"name": "gemv4 16x28672 k4096", "op": "gemv", "fmt": "mxfp4", "m": 16, "n": 28672, "k": 4096, "out": "bf16"},
        # a ragged batch on NVFP4 weights, fp32 results (logits or partial sums of a sharded layer)
        {"name": "gemvnv 5x14336 k4096", "op": "gemv", "fmt": "nvfp4", "m": 5, "n": 14336, "k": 4096, "out": "f32"},
        # the tiny MoE layer, three tokens: latency of the whole layer
        {"name": "decode4 tiny T3", "op": "decode", "fmt": "mxfp4", "tokens": 3, "topk": 2, "experts": 4, "hidden": 256,
         "ffn": 512},
        # one token of the 8-expert layer, 4-bit weights
        {"name": "decode4 T1 e8", "op": "decode", "fmt": "mxfp4", "tokens": 1, "topk": 2, "experts": 8, "hidden": 4096,
         "ffn": 14336},
        # a few tokens on 8-bit weights: most experts are read
        {"name": "decode8 T7 e8", "op": "decode", "fmt": "mxfp8", "tokens": 7, "topk": 2, "experts": 8, "hidden": 4096,
         "ffn": 14336},
        # the largest decoding batch: every expert is read, for many rows each
        {"name": "decode4 T64 e8", "op": "decode", "fmt": "mxfp4", "tokens": 64, "topk": 2, "experts": 8, "hidden": 4096,
         "ffn": 14336},
        # many small experts, master weights in bf16
        {"name": "decode16 T13 e64", "op": "decode", "fmt": "bf16", "tokens": 13, "topk": 6, "experts": 64, "hidden": 2048,
         "ffn": 1024},
        # routing of a decoding batch over many experts
        {"name": "route T33 e128", "op": "route", "tokens": 33, "experts": 128, "topk": 8, "dtype": "bf16", "renorm": True,
         "bias": True},
        # routing of a training step's tokens
        {"name": "route T8192 e8", "op": "route", "tokens": 8192, "experts": 8, "topk": 2, "dtype": "f32", "renorm": True,
         "bias": False},
        # gradient of the router from the experts' dprobs, odd number of tokens, weights not renormalized
        {"name": "route bwd T16383 e128", "op": "route_bwd", "tokens": 16383, "experts": 128, "topk": 8, "dtype": "bf16",
         "renorm": False, "bias": False},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "decode", "decode", "route", "route_bwd"])
    if op == "gemv":
        return {"op": op, "fmt": rng.choice(["mxfp4", "nvfp4"]), "m": _spread(rng, 1, 64), "n": _spread(rng, 16, 32000),
                "k": 32 * _spread(rng, 1, 448), "out": rng.choice(["bf16", "f32"])}
    if op == "decode":
        fmt = rng.choice(["bf16", "mxfp8", "mxfp4"])
        experts = rng.choice([1, 4, 8, 16, 60, 128])
        hidden, ffn = 32 * _spread(rng, 4, 128), 32 * _spread(rng, 4, 448)
        while experts * 3 * hidden * ffn * FORMAT_BYTES[fmt] > 7e8:
            ffn = max(32, ffn // 64 * 32)
            hidden = max(128, hidden // 64 * 32) if ffn <= 128 else hidden
        return {"op": op, "fmt": fmt, "tokens": _spread(rng, 1, 64), "topk": rng.randint(1, min(8, experts)),
                "experts": experts, "hidden": hidden, "ffn": ffn}
    experts = rng.choice([4, 8, 16, 60, 64, 128])
    return {"op": op, "tokens": _spread(rng, 1, 16384), "experts": experts, "topk": rng.randint(1, min(8, experts)),
            "dtype": rng.choice(["bf16", "f32"]), "renorm": rng.random() < 0.5, "bias": rng.random() < 0.5}


# ---- the casts that make the weights

def _e2m1_codes(v):
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    code = torch.bucketize(v.abs(), mid, out_int32=True).to(torch.uint8)
    return code | ((v < 0).to(torch.uint8) << 3)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _cast(w, fmt):
    """w f32 [rows, cols] -> what a program holds: codes and scales (nvfp4: and the tensor's amax)."""
    if fmt == "bf16":
        return (w.to(torch.bfloat16),)
    group = 16 if fmt == "nvfp4" else 32
    v = w.view(w.shape[0], -1, group)
    top = v.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        amax = w.abs().amax().reshape(1)
        big = 2688.0 / amax
        s = (top / 6 * big).clamp(max=448.0).to(torch.float8_e4m3fn)
        sf = s.float()
        codes = _e2m1_codes(torch.where(sf > 0, v * (big / sf), torch.zeros_like(v)))
        return _pack(codes.view(w.shape)), s.view(torch.uint8).squeeze(-1), amax
    e = (torch.frexp(top)[1] - 1 - (8 if fmt == "mxfp8" else 2)).clamp(-126, 127)
    v = torch.ldexp(v, -e)
    s = (e + 127).to(torch.uint8).squeeze(-1)
    if fmt == "mxfp8":
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(w.shape), s
    return _pack(_e2m1_codes(v).view(w.shape)), s


def _weights(gen, experts, rows, cols, fmt):
    parts = [_cast(0.02 * torch.randn((rows, cols), generator=gen, device=DEV), fmt) for _ in range(experts)]
    return [torch.stack(p) for p in zip(*parts)]


def _router_logits(gen, tokens, experts, dtype):
    """Logits of skewed load: a spread per token and one per expert."""
    z = torch.randn((tokens, experts), generator=gen, device=DEV) + 0.7 * torch.randn(experts, generator=gen, device=DEV)
    return z.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "gemv":
        w = _weights(gen, 1, case["n"], case["k"], case["fmt"])
        s["w"] = [t[0] for t in w]
        s["x"] = torch.randn((case["m"], case["k"]), generator=gen, device=DEV).to(torch.bfloat16)
        s["out_dtype"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    elif case["op"] == "decode":
        e, h, f = case["experts"], case["hidden"], case["ffn"]
        s["w1"] = _weights(gen, e, 2 * f, h, case["fmt"])
        s["w2"] = _weights(gen, e, h, f, case["fmt"])
        s["x"] = torch.randn((case["tokens"], h), generator=gen, device=DEV).to(torch.bfloat16)
        z = _router_logits(gen, case["tokens"], e, "f32")
        top, idx = torch.sort(z, dim=1, descending=True, stable=True)
        s["topk_w"] = torch.softmax(top[:, :case["topk"]], 1).contiguous()
        s["topk_idx"] = idx[:, :case["topk"]].to(torch.int32).contiguous()
    else:
        t, e, k = case["tokens"], case["experts"], case["topk"]
        z = _router_logits(gen, t, e, case["dtype"])
        z[torch.rand((t, e), generator=gen, device=DEV) < 0.01] = -math.inf      # a few experts closed to a few tokens
        s["logits"] = z
        s["bias"] = 0.1 * torch.randn(e, generator=gen, device=DEV) if case["bias"] else None
        if case["op"] == "route_bwd":
            idx, w, lse = _route_plain(z, s["bias"], k, case["renorm"])
            s["topk_idx"], s["topk_w"], s["lse"] = idx, w, lse
            # routed rows by expert, then token, as the dispatch numbers them; the entries without an expert have none
            flat = torch.where(idx < 0, torch.full_like(idx, e), idx).reshape(-1)
            order = torch.argsort(flat, stable=True)
            perm = torch.empty(t * k, dtype=torch.int32, device=DEV)
            perm[order] = torch.arange(t * k, dtype=torch.int32, device=DEV)
            s["perm"] = torch.where(idx < 0, torch.full_like(idx, -1), perm.view(t, k))
            s["dprobs"] = 1e-3 * torch.randn(t * k, generator=gen, device=DEV)
    return s


# ---- the plain forms

def _scale_values(s):
    return (s.to(torch.int32) << 23).view(torch.float32)            # 2^(s - 127), s >= 1


def _plain(w, fmt):
    """Block-scaled weights [..., k] in f32."""
    if fmt == "bf16":
        return w[0].float()
    if fmt == "mxfp8":
        v = w[0].view(torch.float8_e4m3fn).float()
        return (v.view(*v.shape[:-1], -1, 32) * _scale_values(w[1]).unsqueeze(-1)).view(v.shape)
    one = torch.tensor(E2M1 + [-a for a in E2M1], device=DEV)
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)          # byte -> its two values
    v = pair[w[0].to(torch.int32)].flatten(-2)
    if fmt == "mxfp4":
        return (v.view(*v.shape[:-1], -1, 32) * _scale_values(w[1]).unsqueeze(-1)).view(v.shape)
    s = w[1].view(torch.float8_e4m3fn).float()
    return (v.view(*v.shape[:-1], -1, 16) * s.unsqueeze(-1)).view(v.shape) / (2688.0 / w[2])


def _route_plain(z, bias, k, renorm):
    z = z.float()
    key = z if bias is None else z + bias
    open_ = key > -math.inf
    key = torch.where(open_, key, torch.full_like(key, -math.inf))
    top, idx = torch.sort(key, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    taken = top > -math.inf
    z = torch.where(open_, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, 1)
    zk = torch.where(taken, torch.gather(z, 1, idx), torch.full_like(top, -math.inf))
    ref = torch.logsumexp(zk, 1) if renorm else lse
    w = torch.where(taken, torch.exp(zk - ref[:, None]), torch.zeros_like(zk))
    return torch.where(taken, idx, -1).to(torch.int32), w, lse


def _run_plain(s):
    if s["op"] == "gemv":
        return (s["x"].float() @ _plain(s["w"], s["fmt"]).T).to(s["out_dtype"])
    if s["op"] == "decode":
        idx, e, f = s["topk_idx"].long(), s["experts"], s["ffn"]
        x = s["x"].float()
        if idx.numel() < e:                                         # fewer choices than experts: the chosen ones' weights
            ids = idx.reshape(-1)
            tokens = torch.arange(idx.shape[0], device=DEV).repeat_interleave(idx.shape[1])
            w1, w2 = _plain([t[ids] for t in s["w1"]], s["fmt"]), _plain([t[ids] for t in s["w2"]], s["fmt"])
            h = torch.bmm(x[tokens].unsqueeze(1), w1.transpose(1, 2))
            a = s["topk_w"].view(-1, 1, 1) * h[..., :f] * torch.sigmoid(h[..., :f]) * h[..., f:]
            y = torch.bmm(a, w2.transpose(1, 2)).view(*idx.shape, -1).sum(1)
        else:
            share = ((idx.unsqueeze(-1) == torch.arange(e, device=DEV)) * s["topk_w"].unsqueeze(-1)).sum(1)     # [T, E]
            h = torch.matmul(x, _plain(s["w1"], s["fmt"]).transpose(1, 2))
            a = share.T.unsqueeze(-1) * h[..., :f] * torch.sigmoid(h[..., :f]) * h[..., f:]
            y = torch.bmm(a, _plain(s["w2"], s["fmt"]).transpose(1, 2)).sum(0)
        return y.to(torch.bfloat16)
    if s["op"] == "route":
        idx, w, lse = _route_plain(s["logits"], s["bias"], s["topk"], s["renorm"])
        return {"idx": idx, "w": w, "lse": lse}
    z, perm, idx = s["logits"].float(), s["perm"].long(), s["topk_idx"].long()
    dw = torch.where(perm >= 0, s["dprobs"][perm.clamp(min=0)], torch.zeros_like(s["topk_w"]))
    dot = (s["topk_w"] * dw).sum(1, keepdim=True)
    own_part = torch.where(idx >= 0, s["topk_w"] * dw, torch.zeros_like(dw))
    dz = torch.zeros_like(z).scatter_add(1, idx.clamp(min=0), own_part)
    if s["renorm"]:
        dz = dz - torch.zeros_like(z).scatter_add(1, idx.clamp(min=0), s["topk_w"] * dot)
    else:
        open_ = (z if s["bias"] is None else z + s["bias"]) > -math.inf
        dz = dz - torch.where(open_, torch.exp(z - s["lse"][:, None]) * dot, torch.zeros_like(z))
    return dz.to(s["logits"].dtype)


def _run_own(s):
    import mxfp8_block_scaled_mx_amd as mx
    if s["op"] == "gemv":
        if s["fmt"] == "mxfp4":
            return mx.mx_gemv_fp4(s["x"], s["w"][0], s["w"][1], out_dtype=s["out_dtype"])
        return mx.mx_gemv_nvfp4(s["x"], s["w"][0], s["w"][1], s["w"][2], out_dtype=s["out_dtype"])
    if s["op"] == "decode":
        w1, w2 = s["w1"], s["w2"]
        if s["fmt"] == "bf16":
            return mx.grouped_mlp_decode(s["x"], s["topk_idx"], s["topk_w"], w1[0], w2[0])
        return mx.grouped_mlp_decode(s["x"], s["topk_idx"], s["topk_w"], w1[0], w2[0], w1[1], w2[1])
    if s["op"] == "route":
        idx, w, lse = mx.mx_moe_route(s["logits"], s["topk"], bias=s["bias"], renormalize=s["renorm"])
        return {"idx": idx, "w": w, "lse": lse}
    return mx.mx_moe_route_bwd(s["logits"], s["topk_idx"], s["topk_w"], s["lse"], s["dprobs"], perm=s["perm"],
                               bias=s["bias"], renormalize=s["renorm"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": n * k * FORMAT_BYTES[case["fmt"]] + 2 * m * k + size * m * n, "flops": 2 * m * n * k}
    t, e, k = case["tokens"], case["experts"], case["topk"]
    if case["op"] == "decode":
        h, f = case["hidden"], case["ffn"]
        read = e * (1 - (1 - k / e) ** t)                           # experts that are chosen, at even odds
        return {"bytes": read * 3 * h * f * FORMAT_BYTES[case["fmt"]] + 4 * t * h + 8 * t * k, "flops": 6 * t * k * h * f}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route":
        return {"bytes": t * e * size + 8 * t * k + 4 * t, "flops": 4 * t * e}
    read = 0 if case["renorm"] else t * (e * size + 4)              # the softmax over all experts needs the logits again
    return {"bytes": read + t * e * size + 16 * t * k, "flops": 4 * t * e}


# ---- the definitions in 64 bits

def _value64(w, fmt, i):
    """Expert i's weights in f64, element by element from the formats' definitions."""
    if fmt == "bf16":
        return w[0][i].double()
    c, s = w[0][i], w[1][i]
    if fmt == "mxfp8":
        mant, expo = (c & 7).double(), ((c >> 3) & 15).int()
        mag = torch.where(expo == 0, torch.ldexp(mant, torch.full_like(expo, -9)), torch.ldexp(8 + mant, expo - 10))
        v = torch.where(c >= 128, -mag, mag)
        return v * torch.pow(2.0, s.double() - 127).repeat_interleave(32, -1)
    nib = torch.empty((*c.shape[:-1], 2 * c.shape[-1]), dtype=torch.uint8, device=c.device)
    nib[..., 0::2], nib[..., 1::2] = c & 15, c >> 4
    mant, expo = (nib & 1).double(), ((nib >> 1) & 3).int()
    mag = torch.where(expo == 0, mant / 2, torch.ldexp(2 + mant, expo - 2))
    v = torch.where(nib >= 8, -mag, mag)
    if fmt == "mxfp4":
        return v * torch.pow(2.0, s.double() - 127).repeat_interleave(32, -1)
    return v * s.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * (w[2][i].double() / 2688)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemv":
        return s["x"].double() @ _value64([t[None] for t in s["w"]], case["fmt"], 0).mT.contiguous()
    if case["op"] == "decode":
        x, f = s["x"].double(), case["ffn"]
        y = torch.zeros_like(x)
        for i in s["topk_idx"].unique().tolist():
            t, j = (s["topk_idx"] == i).nonzero(as_tuple=True)
            h = x[t] @ _value64(s["w1"], case["fmt"], i).mT.contiguous()
            a = h[:, :f] / (1 + torch.exp(-h[:, :f])) * h[:, f:] * s["topk_w"][t, j].double()[:, None]
            y.index_add_(0, t, a @ _value64(s["w2"], case["fmt"], i).mT.contiguous())
        return y
    z, k = s["logits"].double(), case["topk"]
    shut = torch.isinf(z)
    if case["op"] == "route":
        idx = _route_plain(s["logits"], s["bias"], k, case["renorm"])[0].long()
        p = torch.exp(z)
        zk = torch.where(idx >= 0, p.gather(1, idx.clamp(min=0)), torch.zeros((), dtype=z.dtype, device=DEV))
        total = zk.sum(1) if case["renorm"] else p.sum(1)
        return {"idx": None, "w": zk / total[:, None], "lse": torch.log(p.sum(1))}
    # the gradient by autograd through the weights' definition
    z = torch.where(shut, torch.full_like(z, -math.inf), z).requires_grad_()
    idx = s["topk_idx"].long()
    p = torch.exp(z)
    zk = torch.where(idx >= 0, p.gather(1, idx.clamp(min=0)), torch.zeros((), dtype=z.dtype, device=DEV))
    w = zk / (zk.sum(1) if case["renorm"] else p.sum(1))[:, None]
    rows = s["perm"].long()
    dw = torch.where(rows >= 0, s["dprobs"].double()[rows.clamp(min=0)], torch.zeros((), dtype=z.dtype, device=DEV))
    (w * dw).sum().backward()
    return z.grad

"""Cases that measure the operators around the quantized products on a GPU.

Three kinds of pass, each what a prompt or a decode step does between two products:

* ``norm``: the residual stream takes a block's output, is normed (root mean square) and rotated and
  quantized to 4 or 8 bits for the next product; the codes are then decoded to the values that they stand for;
* ``product``: the quantized product with bias, activation and residual in its epilogue;
* ``route``: logits of a router to expert ids and weights.

``run`` computes them in elementary torch operations where ``own`` is false, and through the library's entry
points where it is true.  Codes have to be equal between the two, so the plain forms follow the operators'
order of roundings: fp32 steps, and 64 bits for the sum of squares and for the scores that choices compare.
"""
import math

import numpy as np
import torch

own = False

EPS = float(np.float32(1e-6))
FLOATS = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one new token entering a 5120-wide block: a launch's latency is all there is
        dict(name="norm_token", op="norm", tokens=1, width=5120, dtype="bf16", bits=4, rotation=32, residual=True, pad=0),
        # the attention block's input of a 512-token prompt
        dict(name="norm_attn512", op="norm", tokens=512, width=5120, dtype="bf16", bits=4, rotation=32, residual=True, pad=0),
        # odd: rows of 65 blocks inside a wider buffer, fp32 stream, 8 bits, no rotation, first block (no residual yet)
        dict(name="norm_odd_rows", op="norm", tokens=1333, width=2080, dtype="fp32", bits=8, rotation=0, residual=False, pad=36),
        # prompts of several users batched: the stream is larger than every cache
        dict(name="norm_batch8192", op="norm", tokens=8192, width=5120, dtype="bf16", bits=8, rotation=128, residual=True, pad=0),
        # the output projection of one new token, added into the bf16 stream
        dict(name="product_token", op="product", tokens=1, k=5120, n=5120, bits=4, rotation=32, bias=False, act="none", residual="bf16", out="bf16"),
        # the same of a 512-token prompt
        dict(name="product_attn512", op="product", tokens=512, k=5120, n=5120, bits=4, rotation=32, bias=False, act="none", residual="bf16", out="bf16"),
        # odd: neither the rows nor the columns fill tiles, K ends inside a group of blocks; fp32 stream
        dict(name="product_odd", op="product", tokens=77, k=2080, n=1056, bits=8, rotation=0, bias=True, act="gelu", residual="fp32", out="fp32"),
        # the gate of a 17408-wide feed-forward block over a 1024-token micro-batch
        dict(name="product_long1024", op="product", tokens=1024, k=5120, n=17408, bits=4, rotation=32, bias=True, act="silu", residual="none", out="bf16"),
        # one new token over 128 experts
        dict(name="route_token", op="route", tokens=1, experts=128, topk=8, score="softmax", bias=False, groups=1, kept=1, pair=False, renorm=True, scale=1.0, dtype="fp32"),
        # a 512-token prompt over the same experts
        dict(name="route_moe512", op="route", tokens=512, experts=128, topk=8, score="softmax", bias=False, groups=1, kept=1, pair=False, renorm=True, scale=1.0, dtype="fp32"),
        # an odd batch with groups of experts, sigmoid scores and a bias that balances the load
        dict(name="route_groups", op="route", tokens=4099, experts=256, topk=8, score="sigmoid", bias=True, groups=8, kept=4, pair=True, renorm=True, scale=2.5, dtype="bf16"),
        # the most experts that the expert sort takes, a large batch
        dict(name="route_batch16384", op="route", tokens=16384, experts=512, topk=10, score="softmax", bias=True, groups=1, kept=1, pair=False, renorm=True, scale=1.0, dtype="fp32"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "product", "route"])
    if op == "norm":
        tokens = _log(rng, 1, 8192)
        rotation = rng.choice([0, 32, 64, 128])
        unit = max(32, rotation)
        width = unit * max(1, _log(rng, 32, min(17408, 8192 * 5120 // tokens)) // unit)
        return dict(op=op, tokens=tokens, width=width, dtype=rng.choice(["bf16", "fp32"]) if tokens * width < 16 << 20 else "bf16",
                    bits=rng.choice([4, 8]), rotation=rotation, residual=rng.random() < 0.75, pad=4 * rng.randrange(0, 9) * (rng.random() < 0.5))
    if op == "product":
        tokens = _log(rng, 1, 1024)
        k = 32 * max(1, _log(rng, 32, 17408) // 32)
        n = 32 * max(1, _log(rng, 32, min(17408, 1024 * 5120 * 17408 // (tokens * k))) // 32)
        return dict(op=op, tokens=tokens, k=k, n=n, bits=rng.choice([4, 8]), rotation=32 if k % 64 else rng.choice([0, 32, 64]),
                    bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                    residual=rng.choice(["none", "bf16", "fp32"]), out=rng.choice(["bf16", "fp32"]))
    tokens = _log(rng, 1, 16384)
    groups = rng.choice([1, 1, 2, 4, 8])
    experts = groups * _log(rng, 3 if groups > 1 else 8, 512 // groups)
    kept = groups if groups == 1 else rng.randint(1, groups)
    return dict(op=op, tokens=tokens, experts=experts, topk=rng.randint(1, min(16, kept * (experts // groups))), score=rng.choice(["softmax", "sigmoid"]),
                bias=rng.random() < 0.5, groups=groups, kept=kept, pair=rng.random() < 0.5, renorm=rng.random() < 0.75, scale=rng.choice([1.0, 2.5]),
                dtype=rng.choice(["bf16", "fp32"]))


# ---------------------------------------------------------------- inputs

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _generator(seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=_device(), dtype=torch.float32)


def _outliers(g, x, times):
    """Half a percent of the channels much larger than the rest, as activations have them."""
    k = x.shape[1]
    x[:, torch.randperm(k, generator=g, device=_device())[: max(1, k // 200)]] *= times
    return x


def prepare(case, seed):
    g = _generator(seed)
    state = dict(case)
    if case["op"] == "norm":
        m, k, dtype = case["tokens"], case["width"], FLOATS[case["dtype"]]
        rows = lambda times: _outliers(g, _normal(g, m, k + case["pad"]), times).to(dtype)[:, :k]  # noqa: E731
        state["x"] = rows(30.0)
        state["r"] = rows(10.0) if case["residual"] else None
        state["weight"] = (1.0 + 0.1 * _normal(g, k)).to(dtype)
    elif case["op"] == "product":
        m, k, n, bits = case["tokens"], case["k"], case["n"], case["bits"]
        blocks, groups = k // 32, (k // 32 + 3) // 4
        # activations: normal values, quantized per block of 32
        x = _normal(g, m, blocks, 32)
        state["scales"] = (x.abs().amax(-1) / (7.0 if bits == 4 else 127.0)).contiguous()
        q = (x / state["scales"][..., None]).round().to(torch.int32)
        if bits == 4:
            q = (q[..., :16] & 15) | ((q[..., 16:] & 15) << 4)
        state["codes"] = q.reshape(m, -1).to(torch.int16).bitwise_and(255).to(torch.uint8)
        # the weight image as the packer lays it out: per tile of 32 columns and group of four blocks 2048 bytes of
        # nibbles ([slot][column][block] dwords) and 128 fp16 scales ([16 columns][half][block])
        codes = torch.randint(0, 256, (n // 32, groups, 4, 32, 4, 4), generator=g, device=_device(), dtype=torch.uint8)
        scale = (0.002 + 0.018 * torch.rand(n // 32, groups, 16, 2, 4, generator=g, device=_device())).to(torch.float16)
        past = blocks % 4
        if past:
            codes[:, -1, :, :, past:] = 0x88
            scale[:, -1, :, :, past:] = 0
        state["image"] = torch.cat([codes.view(n // 32, groups, 2048), scale.view(n // 32, groups, 128).view(torch.uint8)], 2).reshape(-1)
        state["bias"] = _normal(g, n) if case["bias"] else None
        state["r"] = None if case["residual"] == "none" else _normal(g, m, n).to(FLOATS[case["residual"]])
    else:
        t, e = case["tokens"], case["experts"]
        state["logits"] = (2.0 * _normal(g, t, e)).to(FLOATS[case["dtype"]])
        state["bias"] = 0.1 * _normal(g, e) if case["bias"] else None
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    return {"norm": _norm, "product": _product, "route": _route}[state["op"]](state)


def _butterflies(v, span):
    """The Sylvester-order Hadamard transform of every span, stage by stage in the input's type, without its factor."""
    shape = v.shape
    h = 1
    while h < span:
        v = v.reshape(-1, 2, h)
        v = torch.stack((v[:, 0] + v[:, 1], v[:, 0] - v[:, 1]), 1)
        h *= 2
    return v.reshape(shape)


def _factor(span):
    return float(np.float32(1.0 / math.sqrt(span)))


def _norm(s):
    x, r, weight, bits, span = s["x"], s["r"], s["weight"], s["bits"], s["rotation"]
    if own:
        from bit_prefill_gemm_amd import binding as bpg
        h, codes, scales = bpg.rmsnorm_quantize_act(x, residual=r, weight=weight, eps=EPS, act_bits=bits, rotation=span)
        values = bpg.dequantize_act(codes, scales, act_bits=bits, rotation=span, dtype=torch.bfloat16)
        return {"scales": scales, "values": values} if r is None else {"h": h, "scales": scales, "values": values}
    m, k = x.shape
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    f = h.float()
    rstd = (1.0 / torch.sqrt(f.double().square().mean(1, keepdim=True) + EPS)).float()
    v = f * rstd * weight.float()
    if span:
        v = _butterflies(v, span) * _factor(span)
    v = v.reshape(m, k // 32, 32)
    top = 7.0 if bits == 4 else 127.0
    amax = v.abs().amax(2, keepdim=True)
    d = amax / torch.full_like(amax, top)
    q = torch.where(d > 0, torch.round(v / d), 0.0).clamp(-top - (bits == 4), top)
    values = (q * d).reshape(m, k)
    if span:
        values = _butterflies(values, span) * _factor(span)
    out = {"scales": d.reshape(m, k // 32), "values": values.to(torch.bfloat16)}
    return out if r is None else {"h": h, **out}


def _stamp(bpg, s):
    """The weights as the library's handle: the stamp that the packer writes, and the image."""
    n, k = s["n"], s["k"]
    stamp = bpg.WeightsDesc(0x57475042, 1, s["rotation"], 3, n, k, 1, (n // 32) * ((k // 32 + 3) // 4) * 2304, 2048)
    return bpg.Weights(stamp, s["image"])


def _decode(s):
    """(activations [m][k], weights [n][k]) in fp32: the values of the codes times their scales."""
    m, n, k = s["tokens"], s["n"], s["k"]
    blocks, groups = k // 32, (k // 32 + 3) // 4
    if s["bits"] == 4:
        c = s["codes"].reshape(m, blocks, 16)
        q = torch.cat([c & 15, c >> 4], 2).to(torch.int8)
        q = torch.where(q > 7, q - 16, q)
    else:
        q = s["codes"].view(torch.int8).reshape(m, blocks, 32)
    a = (q.float() * s["scales"][..., None]).reshape(m, k)
    image = s["image"].view(n // 32, groups, 2304)
    # [tile][group][slot][column][block][byte] -> [tile][column][group][block][slot][byte]
    c = image[..., :2048].reshape(n // 32, groups, 4, 32, 4, 4).permute(0, 3, 1, 4, 2, 5).reshape(n, groups * 4, 16)
    # [tile][group][column % 16][column / 16][block] -> [tile][column / 16][column % 16][group][block]
    d = image[..., 2048:].contiguous().view(torch.float16).reshape(n // 32, groups, 16, 2, 4).permute(0, 3, 2, 1, 4).reshape(n, groups * 4)
    u = torch.cat([c & 15, c >> 4], 2)[:, :blocks]
    w = ((u.float() - 8.0) * d[:, :blocks, None].float()).reshape(n, k)
    return a, w


def _activation(t, act):
    if act == "relu":
        return torch.clamp(t, min=0.0)
    if act == "silu":
        return t / (1.0 + torch.exp(-t))
    if act == "gelu":
        return 0.5 * t * (1.0 + torch.erf(t * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * t * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (t + 0.044715 * t * t * t)))
    return t


def _product(s):
    if own:
        from bit_prefill_gemm_amd import binding as bpg
        return bpg.w4a4_gemm_epilogue(s["codes"], s["scales"], s["bits"], _stamp(bpg, s), bias=s["bias"], activation=s["act"],
                                      residual=s["r"], dtype=FLOATS[s["out"]], rotation=s["rotation"])
    a, w = _decode(s)
    y = torch.mm(a, w.t())
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _activation(y, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(FLOATS[s["out"]])


def _route(s):
    logits, bias, groups, kept, topk = s["logits"], s["bias"], s["groups"], s["kept"], s["topk"]
    if own:
        from bit_prefill_gemm_amd import binding as bpg
        ids, weights = bpg.moe_route_topk(logits, topk, score=s["score"], bias=bias, groups=groups, topk_groups=kept,
                                          group_score="top2" if s["pair"] else "max", renormalize=s["renorm"], scale=s["scale"])
        return {"ids": ids, "weights": weights}
    t, e = logits.shape
    l = logits.double()
    if s["score"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    key = p if bias is None else p + bias.double()
    if groups > 1:
        best = torch.sort(key.view(t, groups, e // groups), dim=2, descending=True).values
        score = best[..., 0] + best[..., 1] if s["pair"] else best[..., 0]
        chosen = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :kept]
        open_ = torch.zeros_like(score, dtype=torch.bool).scatter(1, chosen, True)
        key = torch.where(open_[..., None], key.view(t, groups, e // groups), -math.inf).view(t, e)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk]
    w = torch.gather(p, 1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32).reshape(-1), "weights": (w * s["scale"]).float().reshape(-1)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = {"bf16": 2, "fp32": 4, "none": 0}
    if case["op"] == "norm":
        m, k, e = case["tokens"], case["width"], size[case["dtype"]]
        values = m * k
        return {"bytes": values * (e * (3 if case["residual"] else 1) + 2) + values // 32 * 4 + k * e,
                "flops": values * (12 + 2 * int(math.log2(max(1, case["rotation"]))))}
    if case["op"] == "product":
        m, n, k = case["tokens"], case["n"], case["k"]
        image = (n // 32) * ((k // 32 + 3) // 4) * 2304
        return {"bytes": m * k * case["bits"] // 8 + m * k // 8 + image + n * 4 * case["bias"] + m * n * (size[case["residual"]] + size[case["out"]]),
                "flops": 2 * m * n * k}
    t, e = case["tokens"], case["experts"]
    return {"bytes": t * e * size[case["dtype"]] + e * 4 * case["bias"] + t * case["topk"] * 8, "flops": 8 * t * e}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "product": _exact_product, "route": _exact_route}[case["op"]](s)


def _exact_norm(s):
    x, span, bits = s["x"].double(), s["rotation"], s["bits"]
    out = {}
    if s["r"] is not None:
        out["h"] = x + s["r"].double()
        x = out["h"].to(s["x"].dtype).double()  # the norm is that of the stream as it is stored
    m, k = x.shape
    v = x * s["weight"].double() / torch.sqrt((x * x).sum(1, keepdim=True) / k + EPS)
    if span:
        i = torch.arange(span, device=x.device)
        parity = torch.zeros(span, span, dtype=torch.int64, device=x.device)
        for bit in range(7):
            parity += (i[:, None] >> bit) & (i[None, :] >> bit) & 1
        hadamard = (1.0 - 2.0 * (parity % 2)).double() / math.sqrt(span)
        v = torch.mm(v.reshape(-1, span), hadamard)
    v = v.reshape(-1, 32)
    d = v.abs().max(1).values / (7 if bits == 4 else 127)
    v = torch.round(v / torch.where(d > 0, d, 1.0)[:, None]) * d[:, None]
    if span:
        v = torch.mm(v.reshape(-1, span), hadamard)
    out["scales"] = d.reshape(m, k // 32)
    out["values"] = v.reshape(m, k)
    return out


def _exact_product(s):
    m, n, k = s["tokens"], s["n"], s["k"]
    groups = (k // 32 + 3) // 4
    dev = s["codes"].device
    j = torch.arange(k, device=dev)
    b, i = j // 32, j % 32
    codes = s["codes"].to(torch.int64)
    if s["bits"] == 4:
        q = (codes[:, b * 16 + i % 16] >> (4 * (i // 16))) & 15
        q = q - 16 * (q >= 8).to(torch.int64)
    else:
        q = codes - 256 * (codes >= 128).to(torch.int64)
    a = q.double() * s["scales"].double()[:, b]
    y = torch.empty(m, n, dtype=torch.float64, device=dev)
    for c0 in range(0, n, 1024):
        c = torch.arange(c0, min(n, c0 + 1024), device=dev)[:, None]
        block = ((c // 32) * groups + b // 4) * 2304
        byte = i % 16
        at = block + (((byte // 4) * 32 + c % 32) * 4 + b % 4) * 4 + byte % 4
        u = (s["image"][at].to(torch.int64) >> (4 * (i // 16))) & 15
        at = block + 2048 + (((c % 16) * 2 + (c % 32) // 16) * 4 + b % 4) * 2
        half = s["image"][at].to(torch.int32) + 256 * s["image"][at + 1].to(torch.int32)
        w = (u - 8).double() * half.to(torch.int16).view(torch.float16).double()
        y[:, c0:c0 + c.shape[0]] = torch.mm(a, w.t().contiguous())
    if s["bias"] is not None:
        y += s["bias"].double()
    if s["act"] == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif s["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif s["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    elif s["act"] == "gelu_tanh":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    return y if s["r"] is None else y + s["r"].double()


def _exact_route(s):
    l = s["logits"].double().cpu().numpy()
    t, e = l.shape
    if s["score"] == "softmax":
        p = np.exp(l - l.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    else:
        p = 1.0 / (1.0 + np.exp(-l))
    key = p + (0.0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    if s["groups"] > 1:
        each = np.sort(key.reshape(t, s["groups"], -1), axis=2)
        score = each[:, :, -1] + (each[:, :, -2] if s["pair"] else 0.0)
        out = np.argsort(-score, axis=1, kind="stable")[:, s["kept"]:]
        for column in out.T:
            key.reshape(t, s["groups"], -1)[np.arange(t), column] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, : s["topk"]]
    w = np.take_along_axis(p, ids, 1)
    if s["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return {"ids": None, "weights": (w * s["scale"]).reshape(-1)}

"""Cases that measure the 8-bit floating-point route and the log probabilities of tokens on a GPU.

Four kinds of pass, each what a prompt or a decode step does:

* ``quantize``: rows of activations (or whole weights) to e4m3 codes with a scale per block of 128 (128 x 128);
* ``product``: the product of such codes, every block of 128 under its own scales;
* ``gated``: both projections of a gated feed-forward block, activation and product, as values, or as the codes
  that the down projection reads, with that projection;
* ``logprobs``: log probabilities of given tokens, the entropy of each row of logits and its top alternatives.

``run`` computes them in elementary torch operations where ``own`` is false, and through the library's entry
points where it is true.  Codes are returned as e4m3 values, their scales beside them.
"""
import math

import torch

own = False

FLOATS = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128
TOP = 448.0  # the largest e4m3 value
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one new token entering a 5120-wide block: a launch's latency is all there is
        dict(name="quantize_token", op="quantize", rows=1, width=5120, dtype="bf16", block_rows=1, pad=0),
        # odd: weights whose rows and columns end inside a block, in a wider buffer (made once, when a model is loaded)
        dict(name="quantize_weights_odd", op="quantize", rows=1061, width=2080, dtype="fp32", block_rows=128, pad=36),
        # prompts of several users batched
        dict(name="quantize_batch8192", op="quantize", rows=8192, width=5120, dtype="bf16", block_rows=1, pad=0),
        # the output projection of one new token
        dict(name="product_token", op="product", tokens=1, k=5120, n=5120, out="bf16"),
        # the same of a 512-token prompt
        dict(name="product_attn512", op="product", tokens=512, k=5120, n=5120, out="bf16"),
        # the up projection of several users' prompts batched
        dict(name="product_batch8192", op="product", tokens=8192, k=5120, n=17408, out="bf16"),
        # a whole feed-forward block for one new token: gate and up projection to codes, and the down projection of those
        dict(name="gated_token", op="gated", tokens=1, k=5120, f=17408, act="silu", out="down"),
        # odd: neither rows nor columns fill tiles, K ends inside a block; fp32 values
        dict(name="gated_odd", op="gated", tokens=77, k=2080, f=1061, act="gelu_tanh", out="fp32"),
        # the same block over a 1024-token micro-batch
        dict(name="gated_long1024", op="gated", tokens=1024, k=5120, f=17408, act="silu", out="down"),
        # the answer of one decode step with twenty alternatives
        dict(name="logprobs_token", op="logprobs", tokens=1, vocab=131072, dtype="fp32", topk=20, masked=False),
        # odd: a prompt's tokens scored (perplexity) with five alternatives, part of the vocabulary masked
        dict(name="logprobs_odd", op="logprobs", tokens=333, vocab=50001, dtype="bf16", topk=5, masked=True),
        # several prompts scored at once
        dict(name="logprobs_batch4096", op="logprobs", tokens=4096, vocab=131072, dtype="bf16", topk=1, masked=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(max(low, high))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "gated", "logprobs"])
    if op == "quantize":
        rows = _log(rng, 1, 8192)
        width = 32 * max(1, _log(rng, 32, min(17408, 8192 * 5120 // rows)) // 32)
        small = rows * width < 16 << 20
        return dict(op=op, rows=rows, width=width, dtype=rng.choice(["bf16", "fp32"]) if small else "bf16", block_rows=rng.choice([1, 1, 128]),
                    pad=8 * rng.randrange(0, 9) * (rng.random() < 0.5))
    if op == "product":
        tokens = _log(rng, 1, 8192)
        k = 32 * max(1, _log(rng, 32, 17408) // 32)
        n = _log(rng, 1 if rng.random() < 0.2 else 128, min(17408, 8192 * 5120 * 17408 // (tokens * k)))
        return dict(op=op, tokens=tokens, k=k, n=n, out=rng.choice(["bf16", "fp32"]))
    if op == "gated":
        tokens = _log(rng, 1, 1024)
        k = 32 * max(1, _log(rng, 32, 17408) // 32)
        f = _log(rng, 32, min(17408, 1024 * 5120 * 17408 // (tokens * k)))
        out = rng.choice(["bf16", "fp32", "down"])
        return dict(op=op, tokens=tokens, k=k, f=32 * (f // 32) if out == "down" else f, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]), out=out)
    tokens = _log(rng, 1, 4096)
    vocab = _log(rng, 32, min(262144, 4096 * 131072 // tokens))
    dtype = rng.choice(["bf16", "fp32"]) if tokens * vocab < 128 << 20 else "bf16"
    return dict(op=op, tokens=tokens, vocab=vocab, dtype=dtype, topk=rng.choice([0, 1, 5, 20, 32]), masked=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=_device(), dtype=torch.float32)


def _blocks(k):
    return (k + BLOCK - 1) // BLOCK


def _outliers(g, x, times):
    """Half a percent of the channels much larger than the rest, as activations have them."""
    k = x.shape[1]
    x[:, torch.randperm(k, generator=g, device=_device())[: max(1, k // 200)]] *= times
    return x


def _codes(x, rows):
    """Codes and scales of blocks of `rows` x 128 values, as a checkpoint or an earlier step holds them."""
    m, k = x.shape
    t, b = (m + rows - 1) // rows, _blocks(k)
    padded = torch.zeros(t * rows, b * BLOCK, device=x.device)
    padded[:m, :k] = x
    v = padded.view(t, rows, b, BLOCK)
    d = v.abs().amax((1, 3)) / TOP
    q = (v / torch.where(d > 0, d, 1.0)[:, None, :, None]).to(E4M3)
    return q.view(t * rows, b * BLOCK)[:m, :k].contiguous(), d.contiguous()


def _weights(g, n, k):
    spread = 0.01 + 0.02 * torch.rand(n, 1, generator=g, device=_device())
    return _codes(_normal(g, n, k) * spread, BLOCK)


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    state = dict(case)
    if case["op"] == "quantize":
        m, k = case["rows"], case["width"]
        x = _normal(g, m, k + case["pad"])
        x = _outliers(g, x, 30.0) if case["block_rows"] == 1 else x * 0.02
        state["x"] = x.to(FLOATS[case["dtype"]])[:, :k]
    elif case["op"] == "product":
        state["codes"], state["scales"] = _codes(_outliers(g, _normal(g, case["tokens"], case["k"]), 30.0), 1)
        state["w"] = _weights(g, case["n"], case["k"])
    elif case["op"] == "gated":  # behind a norm, whose weights damp the largest channels
        state["codes"], state["scales"] = _codes(_outliers(g, _normal(g, case["tokens"], case["k"]), 8.0), 1)
        state["gate"] = _weights(g, case["f"], case["k"])
        state["up"] = _weights(g, case["f"], case["k"])
        state["down"] = _weights(g, case["k"], case["f"]) if case["out"] == "down" else None
    else:
        t, v = case["tokens"], case["vocab"]
        logits = _normal(g, t, v)
        logits *= 2.5
        # the token that came is often a likely one; one position in sixteen is padding
        tokens = torch.randint(0, v, (t,), generator=g, device=_device())
        lift = 12.0 * torch.rand(t, 1, generator=g, device=_device())
        logits.scatter_add_(1, tokens[:, None], lift)
        if case["masked"]:
            out = torch.rand(v, generator=g, device=_device()) < 0.25
            logits.masked_fill_(out, -math.inf)
        skip = torch.rand(t, generator=g, device=_device()) < 1 / 16
        state["tokens"] = torch.where(skip, -1, tokens)
        state["logits"] = logits.to(FLOATS[case["dtype"]])
        state["count"] = t
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    return {"quantize": _quantize, "product": _product, "gated": _gated, "logprobs": _logprobs}[state["op"]](state)


def _to_codes(v):
    """fp32 blocks [..., rows, blocks, 128] to (e4m3 codes, scales): d = max / 448, code = e4m3(v (1 / d))."""
    amax = v.abs().amax((-3, -1), keepdim=True)
    d = amax / torch.full_like(amax, TOP)
    r = torch.where(d > 0, 1.0 / d, 0.0)
    return (v * r).to(E4M3), d


def _padded(x, rows):
    m, k = x.shape
    t, b = (m + rows - 1) // rows, _blocks(k)
    if t * rows != m or b * BLOCK != k:
        x = torch.nn.functional.pad(x, (0, b * BLOCK - k, 0, t * rows - m))
    return x.reshape(t, rows, b, BLOCK)


def _quantized(f, rows):
    m, k = f.shape
    q, d = _to_codes(_padded(f, rows))
    return {"codes": q.reshape(-1, _blocks(k) * BLOCK)[:m, :k].contiguous(), "scales": d.reshape(-1, _blocks(k))}


def _quantize(s):
    if own:
        from bit_prefill_gemm_amd import binding as bpg
        codes, scales = bpg.quantize_fp8(s["x"], block_rows=s["block_rows"])
        return {"codes": codes, "scales": scales}
    return _quantized(s["x"].float(), s["block_rows"])


def _values(codes, scales, rows):
    """The fp32 values that codes and scales stand for."""
    n, k = codes.shape
    wide = scales.repeat_interleave(rows, 0)[:n] if rows > 1 else scales
    return codes.float() * wide.repeat_interleave(BLOCK, 1)[:, :k]


def _product(s):
    if own:
        from bit_prefill_gemm_amd import binding as bpg
        return bpg.fp8_gemm(s["codes"], s["scales"], bpg.Fp8Weights(*s["w"]), dtype=FLOATS[s["out"]])
    y = torch.mm(_values(s["codes"], s["scales"], 1), _values(*s["w"], BLOCK).t())
    return y.to(FLOATS[s["out"]])


def _activation(t, act):
    if act == "relu":
        return torch.clamp(t, min=0.0)
    if act == "silu":
        return t / (1.0 + torch.exp(-t))
    if act == "gelu":
        return 0.5 * t * (1.0 + torch.erf(t * math.sqrt(0.5)))
    return 0.5 * t * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (t + 0.044715 * t * t * t)))


def _gated(s):
    if own:
        from bit_prefill_gemm_amd import binding as bpg
        gate, up = bpg.Fp8Weights(*s["gate"]), bpg.Fp8Weights(*s["up"])
        if s["out"] == "down":
            codes, scales = bpg.fp8_gemm_gated_quantize(s["codes"], s["scales"], gate, up, activation=s["act"])
            return bpg.fp8_gemm(codes, scales, bpg.Fp8Weights(*s["down"]), dtype=torch.bfloat16)
        return bpg.fp8_gemm_gated(s["codes"], s["scales"], gate, up, activation=s["act"], dtype=FLOATS[s["out"]])
    a = _values(s["codes"], s["scales"], 1)
    h = _activation(torch.mm(a, _values(*s["gate"], BLOCK).t()), s["act"]) * torch.mm(a, _values(*s["up"], BLOCK).t())
    if s["out"] != "down":
        return h.to(FLOATS[s["out"]])
    q = _quantized(h, 1)
    return torch.mm(_values(q["codes"], q["scales"], 1), _values(*s["down"], BLOCK).t()).to(torch.bfloat16)


def _logprobs(s):
    logits, tokens, topk = s["logits"], s["tokens"], s["topk"]
    if own:
        from bit_prefill_gemm_amd import binding as bpg
        logprobs, entropy, ids, top = bpg.token_logprobs(logits, tokens, topk=topk)
    else:
        f = logits.float()
        shifted = f - f.amax(1, keepdim=True)
        p = torch.exp(shifted)
        # sums over a whole vocabulary: 64 bits
        total = p.sum(1, dtype=torch.float64)
        mean = torch.where(p > 0, shifted * p, 0.0).sum(1, dtype=torch.float64) / total
        entropy = (torch.log(total) - mean).float()
        picked = torch.gather(shifted, 1, tokens.clamp(min=0)[:, None])[:, 0].double()
        logprobs = torch.where(tokens < 0, 0.0, picked - torch.log(total)).float()
        # equal logits: the lowest id first
        order = torch.sort(f, dim=1, descending=True, stable=True).indices[:, :topk]
        ids = order.to(torch.int32)
        top = (torch.gather(shifted, 1, order).double() - torch.log(total)[:, None]).float()
    out = {"logprobs": logprobs, "entropy": entropy}
    return {**out, "ids": ids, "top": top} if topk else out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "quantize":
        m, k, rows = case["rows"], case["width"], case["block_rows"]
        return {"bytes": m * k * (size[case["dtype"]] + 1) + 4 * ((m + rows - 1) // rows) * _blocks(k), "flops": 4 * m * k}
    if case["op"] == "product":
        m, k, n = case["tokens"], case["k"], case["n"]
        return {"bytes": (m + n) * k + 4 * (m + _blocks(n)) * _blocks(k) + m * n * size[case["out"]], "flops": 2 * m * n * k}
    if case["op"] == "gated":
        m, k, f = case["tokens"], case["k"], case["f"]
        down = case["out"] == "down"
        out = k * f + 4 * _blocks(k) * _blocks(f) + 2 * m * k if down else m * f * size[case["out"]]
        return {"bytes": (m + 2 * f) * k + 4 * (m + 2 * _blocks(f)) * _blocks(k) + out, "flops": (6 if down else 4) * m * f * k}
    t, v = case["tokens"], case["vocab"]
    return {"bytes": t * v * size[case["dtype"]] + t * 16 + t * case["topk"] * 8, "flops": 6 * t * v}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "product": _exact_product, "gated": _exact_gated, "logprobs": _exact_logprobs}[case["op"]](s)


def _block_max(v, rows):
    """max |v| of every block [ceil(m / rows)][ceil(k / 128)]."""
    m, k = v.shape
    i = torch.arange(m, device=v.device) // rows
    columns = torch.stack([v[:, j:j + BLOCK].abs().amax(1) for j in range(0, k, BLOCK)], 1)
    out = torch.zeros(int(i[-1]) + 1, columns.shape[1], dtype=v.dtype, device=v.device)
    return out.scatter_reduce(0, i[:, None].expand_as(columns), columns, "amax")


def _exact_codes(v, rows):
    """Scales, and the values that the codes round, both unrounded."""
    m, k = v.shape
    d = _block_max(v, rows) / TOP
    at = d[(torch.arange(m, device=v.device) // rows)[:, None], (torch.arange(k, device=v.device) // BLOCK)[None, :]]
    return {"codes": v / torch.where(at > 0, at, 1.0), "scales": d}


def _exact_quantize(s):
    return _exact_codes(s["x"].double(), s["block_rows"])


def _exact_mm(codes, scales, w):
    """sum over blocks of (x scale) (w scale) (dot product of the codes), in 64 bits."""
    a, (b, e) = codes.double(), w
    y = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    column = torch.arange(b.shape[0], device=a.device) // BLOCK
    for j in range(scales.shape[1]):
        at = slice(j * BLOCK, (j + 1) * BLOCK)
        left = a[:, at] * scales[:, j].double()[:, None]  # scales: fp32, or 64 bits
        right = b[:, at].double() * e[:, j].double()[column][:, None]
        y.addmm_(left, right.t())
    return y


def _exact_product(s):
    return _exact_mm(s["codes"], s["scales"], s["w"])


def _exact_gated(s):
    g, u = _exact_mm(s["codes"], s["scales"], s["gate"]), _exact_mm(s["codes"], s["scales"], s["up"])
    if s["act"] == "relu":
        g = torch.where(g > 0, g, 0.0)
    elif s["act"] == "silu":
        g = g * torch.sigmoid(g)
    elif s["act"] == "gelu":
        g = g * torch.special.ndtr(g)
    else:
        g = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    h = g * u
    if s["out"] != "down":
        return h
    q = _exact_codes(h, 1)  # the codes are a part of the definition
    return _exact_mm(q["codes"].to(E4M3), q["scales"], s["down"])


def _exact_logprobs(s):
    t, topk = s["count"], s["topk"]
    out = {"logprobs": [], "entropy": [], "top": []}
    for a in range(0, t, 256):  # 64-bit rows of a whole vocabulary are large
        l = s["logits"][a:a + 256].double()
        tokens = s["tokens"][a:a + 256]
        z = torch.logsumexp(l, 1, keepdim=True)
        p = torch.exp(l - z)
        out["entropy"].append(torch.special.entr(p).sum(1))
        at = (l - z)[torch.arange(l.shape[0], device=l.device), tokens.clamp(min=0)]
        out["logprobs"].append(torch.where(tokens < 0, 0.0, at))
        out["top"].append(torch.topk(l, topk, dim=1).values - z)
    out = {name: torch.cat(parts) for name, parts in out.items()}
    if not topk:
        del out["top"]
        return out
    return {**out, "ids": None}

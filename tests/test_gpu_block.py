"""The operators between the products run together, as a pre-norm block uses them:

  dense half:   residual addition + norm + quantize -> product with bias and
                activation -> quantize -> product added into the stream
  expert half:  residual addition + norm + quantize -> router logits (a product)
                -> routing -> expert sort -> gathered gate/up -> SwiGLU-quantize
                -> down -> combine

each stage checked against the oracle or a plain 64-bit evaluation on the GPU's
own input to it; the whole chain replayed from a captured graph, issued on
streams of its own, and from two host threads.
"""
import threading

import numpy as np
import pytest

import oracle
from bit_prefill_gemm_amd import binding as bb
from bit_prefill_gemm_amd import synth

from gpu_util import act_to_device, fp32_bound, oracle_codes, torch_mod, weights_to_device
from test_gpu_graph import replay_and_check
from test_gpu_norm import expected, f32, host, quantized
from test_gpu_route import reference

pytestmark = pytest.mark.gpu

H, I, E, TOPK = 512, 160, 32, 4


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    return t


class Block:
    """Weights and inputs of one block over `tokens` tokens."""

    def __init__(self, tokens, bits, seed):
        torch = torch_mod()
        rng = np.random.default_rng(seed)
        self.tokens, self.bits = tokens, bits
        self.x = act_to_device(synth.bf16_bits(rng.standard_normal((tokens, H)).astype(np.float32)))
        self.stream = act_to_device(synth.bf16_bits(2 * rng.standard_normal((tokens, H)).astype(np.float32)))
        self.g = act_to_device(synth.bf16_bits(1 + 0.1 * rng.standard_normal((2, H)).astype(np.float32)))
        self.blocks = {
            "up": synth.draw_q4_0(rng, (3 * H,), H, 0.002, 0.02),
            "down": synth.draw_q4_0(rng, (H,), 3 * H, 0.002, 0.02),
            "router": synth.draw_q4_0(rng, (E,), H, 0.002, 0.02),
            "gu": synth.draw_q4_0(rng, (E * 2 * I,), H, 0.002, 0.02),
            "dn": synth.draw_q4_0(rng, (E * H,), I, 0.002, 0.02),
        }
        self.up = weights_to_device(self.blocks["up"], 3 * H, H)
        self.down = weights_to_device(self.blocks["down"], H, 3 * H)
        self.router = weights_to_device(self.blocks["router"], E, H)
        self.gu = weights_to_device(self.blocks["gu"], 2 * I, H, E)
        self.dn = weights_to_device(self.blocks["dn"], H, I, E)
        self.bias = torch.from_numpy(rng.standard_normal(3 * H).astype(np.float32)).cuda()
        self.balance = torch.from_numpy((0.05 * rng.standard_normal(E)).astype(np.float32)).cuda()

    def dense(self):
        torch = torch_mod()
        h, c1, s1 = bb.rmsnorm_quantize_act(self.x, residual=self.stream, weight=self.g[0], act_bits=self.bits)
        u = bb.w4a4_gemm_epilogue(c1, s1, self.bits, self.up, bias=self.bias, activation="gelu_tanh",
                                  dtype=torch.bfloat16)
        c2, s2 = bb.quantize_act_h32(u, self.bits)
        out = bb.w4a4_gemm_epilogue(c2, s2, self.bits, self.down, residual=h, dtype=torch.bfloat16)
        return [h, c1, s1, u, c2, s2, out]

    def experts(self):
        h, c, s = bb.rmsnorm_quantize_act(self.x, residual=self.stream, weight=self.g[1], act_bits=self.bits)
        logits = bb.w4a4_gemm_epilogue(c, s, self.bits, self.router)
        ids, w = bb.moe_route_topk(logits, TOPK, score="sigmoid", bias=self.balance, groups=8, topk_groups=3,
                                   scale=2.5)
        off, row_token, slot_of = bb.moe_route_sort(ids, self.tokens, TOPK, E)
        gu = bb.w4a4_grouped_gemm_gather(c, s, self.bits, row_token, off, self.gu)
        hc, hs = bb.swiglu_quantize_h32(gu, I, self.bits)
        dn = bb.w4a4_grouped_gemm(hc, hs, self.bits, off, self.dn)
        y = bb.moe_combine(dn, slot_of, w, self.tokens, TOPK)
        return [h, c, s, logits, ids, w, off, row_token, slot_of, gu, hc, hs, dn, y]


def unpack(codes, bits):
    """Code values of the GPU's bytes."""
    c = codes.cpu().numpy()
    if bits == 8:
        return c.view(np.int8)
    m = c.shape[0]
    c = c.reshape(m, -1, 16)
    q = np.concatenate([c & 15, c >> 4], axis=2).astype(np.int8)
    return np.where(q > 7, q - 16, q).astype(np.int8).reshape(m, -1)


def product64(codes, scales, bits, blocks, k):
    q, d = unpack(codes, bits), scales.cpu().numpy()
    w, dw = oracle.q4_0_decode(blocks, k)
    return (oracle.gemm_rect(q, d, w, dw, 0, q.shape[0], 0, w.shape[0]),
            oracle.gemm_abs_rect(q, d, w, dw, 0, q.shape[0], 0, w.shape[0]))


@pytest.mark.parametrize("tokens,bits", [(1, 4), (37, 4), (300, 4), (37, 8)])
def test_dense_half(torch, tokens, bits):
    b = Block(tokens, bits, tokens + bits)
    h, c1, s1, u, c2, s2, out = b.dense()
    ref_h, v = expected(host(b.x), host(b.stream), host(b.g)[0], 1e-6)
    q, d = quantized(v, bits, 32)
    assert np.array_equal(host(h), ref_h)
    assert np.array_equal(host(c1), oracle_codes(q, bits)) and np.array_equal(host(s1), d)
    t, mag = product64(c1, s1, bits, b.blocks["up"], H)
    t = t + b.bias.cpu().numpy().astype(np.float64)
    ref = 0.5 * t * (1 + np.tanh(np.sqrt(2 / np.pi) * (t + 0.044715 * t ** 3)))
    # the product's bound and the bias's rounding through a slope of at most 1.13, the
    # activation's own steps, bf16's half step
    lim = 1.13 * (fp32_bound(mag, H) + 2.0 ** -24 * np.abs(t)) + 12 * 2.0 ** -24 * np.abs(t)
    lim = lim + 2.0 ** -8 * (np.abs(ref) + lim)
    assert (np.abs(f32(host(u)) - ref) <= lim).all()
    q2, d2, _ = oracle.quantize(host(u), bits)
    assert np.array_equal(host(c2), oracle_codes(q2, bits)) and np.array_equal(host(s2), d2)
    t, mag = product64(c2, s2, bits, b.blocks["down"], 3 * H)
    ref = t + f32(ref_h)
    lim = fp32_bound(mag, 3 * H) * (1 + 2.0 ** -16) + 2.0 ** -24 * np.abs(ref)
    lim = lim + 2.0 ** -8 * (np.abs(ref) + lim)
    assert (np.abs(f32(host(out)) - ref) <= lim).all()


@pytest.mark.parametrize("tokens,bits", [(1, 4), (45, 4), (45, 8)])
def test_expert_half(torch, tokens, bits):
    b = Block(tokens, bits, 7 * tokens + bits)
    h, c, s, logits, ids, w, off, row_token, slot_of, gu, hc, hs, dn, y = b.experts()
    ref_h, v = expected(host(b.x), host(b.stream), host(b.g)[1], 1e-6)
    q, d = quantized(v, bits, 32)
    assert np.array_equal(host(c), oracle_codes(q, bits)) and np.array_equal(host(s), d)
    ref, mag = product64(c, s, bits, b.blocks["router"], H)
    assert (np.abs(host(logits) - ref) <= fp32_bound(mag, H) * (1 + 2.0 ** -20)).all()
    ref_ids, ref_w = reference(host(logits), TOPK, "sigmoid", host(b.balance), 8, 3, True, True, 2.5)
    assert np.array_equal(host(ids).reshape(tokens, TOPK), ref_ids)
    assert (np.abs(host(w).reshape(tokens, TOPK) - ref_w) <= (2.0 ** -24 + 2.0 ** -45) * ref_w).all()
    # behind the routing: the layer that the framework had, on these ids and weights
    ref_off, ref_entry, ref_slot = oracle.route_sort(host(ids), E)
    assert np.array_equal(host(off), ref_off) and np.array_equal(host(slot_of), ref_slot)
    assert np.array_equal(host(row_token), ref_entry // TOPK)
    qh, dh, _ = oracle.swiglu_quantize(host(gu), I, bits)
    assert np.array_equal(host(hc), oracle_codes(qh, bits)) and np.array_equal(host(hs), dh)
    ref_y = oracle.moe_combine(host(dn), host(slot_of), host(w), tokens, TOPK)
    assert np.array_equal(host(y), ref_y)


def clear(outs):
    torch = torch_mod()
    for t in outs:
        if t.is_floating_point():
            t.fill_(float("nan"))
        else:
            t.zero_()


@pytest.mark.parametrize("half", ["dense", "experts"])
@pytest.mark.parametrize("tokens,bits", [(1, 4), (70, 8), (600, 4)])
def test_replayed_from_a_graph(torch, half, tokens, bits):
    b, other = Block(tokens, bits, 3), Block(tokens, bits, 4)
    refs = [t.clone() for t in getattr(b, half)()]
    torch.cuda.synchronize()
    replay_and_check(torch, getattr(b, half), getattr(other, half), clear, refs,
                     [str(i) for i in range(len(refs))], "%s %d tokens" % (half, tokens))


def same(a, b):
    return all(torch_mod().equal(x, y) for x, y in zip(a, b))


def test_on_streams_of_their_own(torch):
    """Issued under a stream, with stream=, and from two host threads at once."""
    blocks = [Block(130, 4, 11), Block(90, 8, 12)]
    refs = [[t.clone() for t in b.dense() + b.experts()] for b in blocks]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = blocks[0].dense() + blocks[0].experts()
    s.synchronize()
    assert same(got, refs[0])

    b = blocks[0]
    h, c, sc = bb.rmsnorm_quantize_act(b.x, residual=b.stream, weight=b.g[0], stream=s)
    u = bb.w4a4_gemm_epilogue(c, sc, 4, b.up, bias=b.bias, activation="gelu_tanh", dtype=torch.bfloat16, stream=s)
    v = bb.dequantize_act(c, sc, stream=s)
    ids, w = bb.moe_route_topk(u[:, :64], 5, stream=s)
    s.synchronize()
    assert same([h, c, sc, u], refs[0][:4])
    assert torch.equal(v, bb.dequantize_act(c, sc))
    assert same([ids, w], bb.moe_route_topk(u[:, :64], 5))

    results = [None, None]

    def work(i):
        own = torch.cuda.Stream()
        with torch.cuda.stream(own):
            for _ in range(20):
                results[i] = blocks[i].dense() + blocks[i].experts()
        own.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for got, ref in zip(results, refs):
        assert same(got, ref)


def test_a_stream_of_another_device_is_refused(torch):
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="stream is on"):
        bb.rmsnorm_quantize_act(x, stream=torch.cuda.Stream())


def test_inside_inference_mode_and_with_gradients_asked(torch):
    b = Block(5, 4, 20)
    ref = b.dense()
    with torch.inference_mode():
        assert same(b.dense(), ref)
    x = b.x.float().requires_grad_(True)
    h, codes, scales = bb.rmsnorm_quantize_act(x)
    assert not scales.requires_grad and h is x

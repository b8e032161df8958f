"""Refusals of the 8-bit floating-point route and of token_logprobs: the C ABI
reports every argument error from the host before any HIP call, and the binding
checks every tensor first.  Pointers of the ABI tests are never dereferenced.
"""
import ctypes

import pytest
import torch

from bit_prefill_gemm_amd import binding as bb

OK, NULL, SHAPE, ALIGN, DTYPE, BUFFER, DEVICE = 0, 1, 2, 3, 4, 6, 7
P = ctypes.c_void_p(0x100000)
MIS = ctypes.c_void_p(0x100004)
ODD = ctypes.c_void_p(0x100002)
BYTE = ctypes.c_void_p(0x100001)
NUL = ctypes.c_void_p(0)
E4M3 = torch.float8_e4m3fn

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls would run")


# ------------------------------------------------------------------ C ABI

def quantize(x=P, dt=0, m=4, k=160, ldx=160, rows=1, codes=P, scales=P):
    return bb.lib().quantize_fp8(x, dt, m, k, ldx, rows, codes, scales, NUL)


@pytest.mark.parametrize("args,status", [
    (dict(dt=2), DTYPE), (dict(dt=-1), DTYPE), (dict(rows=0), SHAPE), (dict(rows=64), SHAPE),
    (dict(m=-1), SHAPE), (dict(m=1 << 31), SHAPE), (dict(k=0, ldx=0), SHAPE), (dict(k=48), SHAPE),
    (dict(k=(1 << 22) + 32, ldx=1 << 23), SHAPE), (dict(ldx=159), SHAPE), (dict(ldx=128), SHAPE),
    (dict(m=1 << 30), SHAPE), (dict(m=(1 << 22) + 1, rows=128), SHAPE),
    (dict(x=NUL), NULL), (dict(codes=NUL), NULL), (dict(scales=NUL), NULL),
    (dict(x=MIS), ALIGN), (dict(codes=MIS), ALIGN), (dict(scales=ODD), ALIGN),
    (dict(ldx=162), ALIGN),
])
def test_quantize_abi_refusals(args, status):
    assert quantize(**args) == status


@no_gpu
@pytest.mark.parametrize("args", [
    {}, dict(rows=128), dict(dt=1), dict(m=0, x=NUL, codes=NUL, scales=NUL), dict(scales=MIS),
    dict(k=1 << 22, ldx=1 << 22, m=65535), dict(m=1 << 22, rows=128),
])
def test_quantize_abi_valid_calls_reach_the_device_check(args):
    assert quantize(**args) == DEVICE


def product(codes=P, scales=P, m=4, w=P, ws=P, n=70, k=160, y=P, dt=0, ldy=70, work=P, size=1 << 62):
    return bb.lib().fp8_gemm(codes, scales, m, w, ws, n, k, y, dt, ldy, work, size, NUL)


PRODUCT = [
    (dict(dt=2), DTYPE), (dict(m=-1), SHAPE), (dict(m=(1 << 22) + 1), SHAPE), (dict(n=0), SHAPE),
    (dict(n=(1 << 22) + 1, ldy=1 << 23), SHAPE), (dict(k=0), SHAPE), (dict(k=100), SHAPE),
    (dict(k=(1 << 22) + 32), SHAPE), (dict(ldy=69), SHAPE), (dict(ldy=(1 << 40) + 1), SHAPE),
    (dict(codes=NUL), NULL), (dict(scales=NUL), NULL), (dict(w=NUL), NULL), (dict(ws=NUL), NULL),
    (dict(y=NUL), NULL), (dict(m=0, w=NUL), NULL), (dict(codes=MIS), ALIGN),
    (dict(scales=ODD), ALIGN), (dict(w=MIS), ALIGN), (dict(ws=MIS), ALIGN), (dict(y=ODD), ALIGN),
    (dict(y=BYTE, dt=1), ALIGN),
]


@pytest.mark.parametrize("args,status", PRODUCT + [(dict(work=MIS), ALIGN)])
def test_product_abi_refusals(args, status):
    assert product(**args) == status


@no_gpu
@pytest.mark.parametrize("args", [
    {}, dict(dt=1, y=ODD), dict(y=MIS), dict(scales=MIS), dict(ldy=71), dict(n=1, ldy=1),
    dict(m=0, codes=NUL, scales=NUL, y=NUL), dict(m=1 << 22, k=1 << 22),
])
def test_product_abi_valid_calls_reach_the_device_check(args):
    assert product(**args) == DEVICE


@pytest.mark.parametrize("m,n,k,dt", [(4, 70, 160, 0), (512, 5120, 17408, 1), (1024, 5120, 17408, 1),
                                      (300, 300, 4096, 1), (0, 64, 64, 1)])
def test_product_workspace(m, n, k, dt):
    need = bb.lib().fp8_gemm_bytes(m, n, k, dt)
    args = dict(m=m, n=n, k=k, dt=dt, ldy=n)
    if need:
        assert product(size=need - 1, **args) == BUFFER
        assert product(size=need, work=NUL, **args) == NULL
    if not torch.cuda.is_available():
        assert product(size=need, **args) == DEVICE
        if not need:
            assert product(size=0, work=NUL, **args) == DEVICE
    assert need or (n, k, dt) != (5120, 17408, 1)
    for bad in ((-1, n, k, dt), (m, 0, k, dt), (m, n, 31, dt), (m, n, k, 2)):
        assert bb.lib().fp8_gemm_bytes(*bad) == 0


def gated(codes=P, scales=P, m=4, w=P, ws=P, u=P, us=P, n=96, k=160, act=2, y=P, dt=0, ldy=96):
    return bb.lib().fp8_gemm_gated(codes, scales, m, w, ws, u, us, n, k, act, y, dt, ldy, NUL)


@pytest.mark.parametrize("args,status", PRODUCT + [
    (dict(act=5), DTYPE), (dict(act=-1), DTYPE), (dict(u=NUL), NULL), (dict(us=NUL), NULL),
    (dict(u=MIS), ALIGN), (dict(us=MIS), ALIGN),
])
def test_gated_abi_refusals(args, status):
    assert gated(**args) == status


@no_gpu
@pytest.mark.parametrize("args", [{}, dict(act=0, dt=1), dict(n=97, ldy=97)])
def test_gated_abi_valid_calls_reach_the_device_check(args):
    assert gated(**args) == DEVICE


def gated_quantize(codes=P, scales=P, m=4, w=P, ws=P, u=P, us=P, n=96, k=160, act=2, oc=P, os=P,
                   work=P, size=1 << 62):
    return bb.lib().fp8_gemm_gated_quantize(codes, scales, m, w, ws, u, us, n, k, act, oc, os, work,
                                            size, NUL)


@pytest.mark.parametrize("args,status", [
    (dict(act=5), DTYPE), (dict(m=-1), SHAPE), (dict(n=97), SHAPE), (dict(n=0), SHAPE),
    (dict(k=33), SHAPE), (dict(m=1 << 22, n=1 << 22), SHAPE),
    (dict(codes=NUL), NULL), (dict(u=NUL), NULL), (dict(us=NUL), NULL), (dict(oc=NUL), NULL),
    (dict(os=NUL), NULL), (dict(oc=MIS), ALIGN), (dict(os=ODD), ALIGN), (dict(work=MIS), ALIGN),
])
def test_gated_quantize_abi_refusals(args, status):
    assert gated_quantize(**args) == status


@pytest.mark.parametrize("m,n,k", [(1, 96, 160), (5, 17408, 5120), (300, 640, 320), (64, 32, 32)])
def test_gated_quantize_workspace(m, n, k):
    need = bb.lib().fp8_gemm_gated_quantize_bytes(m, n, k)
    if need:
        assert gated_quantize(m=m, n=n, k=k, size=need - 1) == BUFFER
        assert gated_quantize(m=m, n=n, k=k, size=need, work=NUL) == NULL
    if not torch.cuda.is_available():
        assert gated_quantize(m=m, n=n, k=k, size=need) == DEVICE
        assert gated_quantize(m=0, n=n, k=k, size=0, work=NUL, codes=NUL, scales=NUL, oc=NUL,
                              os=NUL) == DEVICE
    for bad in ((-1, n, k), (m, 0, k), (m, n, 0), (1 << 40, n, k)):
        assert bb.lib().fp8_gemm_gated_quantize_bytes(*bad) == 0


def logprobs(logits=P, dt=0, rows=4, vocab=1000, ldl=1000, tokens=P, tdt=1, topk=5, lp=P, ent=P,
             ids=P, top=P, work=P, size=1 << 62):
    return bb.lib().token_logprobs(logits, dt, rows, vocab, ldl, tokens, tdt, topk, lp, ent, ids, top,
                                   work, size, NUL)


@pytest.mark.parametrize("args,status", [
    (dict(dt=2), DTYPE), (dict(tdt=2), DTYPE), (dict(tdt=-1), DTYPE), (dict(rows=-1), SHAPE),
    (dict(rows=1 << 31), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=(1 << 24) + 1, ldl=1 << 25), SHAPE),
    (dict(ldl=999), SHAPE), (dict(ldl=(1 << 40) + 1), SHAPE), (dict(topk=-1), SHAPE),
    (dict(topk=65), SHAPE), (dict(topk=4, vocab=3), SHAPE), (dict(rows=(1 << 31) - 1, topk=2), SHAPE),
    (dict(logits=NUL), NULL), (dict(lp=NUL), NULL), (dict(ids=NUL), NULL), (dict(top=NUL), NULL),
    (dict(logits=ODD), ALIGN), (dict(logits=BYTE, dt=1), ALIGN), (dict(tokens=MIS), ALIGN),
    (dict(tokens=ODD, tdt=0), ALIGN), (dict(lp=ODD), ALIGN), (dict(ent=ODD), ALIGN),
    (dict(ids=ODD), ALIGN), (dict(top=ODD), ALIGN), (dict(work=MIS), ALIGN),
])
def test_logprobs_abi_refusals(args, status):
    assert logprobs(**args) == status


@no_gpu
@pytest.mark.parametrize("args", [
    {}, dict(tokens=NUL, lp=NUL, tdt=9), dict(ent=NUL), dict(topk=0, ids=NUL, top=NUL),
    dict(tokens=MIS, tdt=0), dict(logits=ODD, dt=1), dict(vocab=1, topk=1),
    dict(rows=0, logits=NUL, tokens=NUL, lp=NUL, ids=NUL, top=NUL, work=NUL, size=0),
])
def test_logprobs_abi_valid_calls_reach_the_device_check(args):
    assert logprobs(**args) == DEVICE


@pytest.mark.parametrize("rows,vocab,topk", [(1, 131072, 20), (4, 1000, 5), (1, 1 << 24, 64), (3, 1, 1)])
def test_logprobs_workspace(rows, vocab, topk):
    need = bb.lib().token_logprobs_bytes(rows, vocab, topk)
    args = dict(rows=rows, vocab=vocab, ldl=vocab, topk=topk)
    if need:
        assert logprobs(size=need - 1, **args) == BUFFER
        assert logprobs(size=need, work=NUL, **args) == NULL
    if not torch.cuda.is_available():
        assert logprobs(size=need, **args) == DEVICE
    for bad in ((-1, vocab, topk), (1 << 31, vocab, topk), (rows, 0, topk), (rows, 1 << 25, topk),
                (rows, vocab, 65), (rows, vocab, -1)):
        assert bb.lib().token_logprobs_bytes(*bad) == 0


# ------------------------------------------------------------------ routing

def test_kernel_names_refuse_what_the_calls_refuse():
    lib = bb.lib()
    for bad in ((-1, 64, 64, 0, 0), (4, 0, 64, 0, 0), (4, 64, 48, 0, 0), (4, 64, 64, 2, 0),
                (1 << 22, 1 << 22, 64, 0, 1)):
        assert lib.fp8_gemm_kernel_name(*bad) is None
    for bad in ((-1, 64, 64), (4, 33, 64), (4, 64, 0)):
        assert lib.fp8_gemm_gated_quantize_kernel_name(*bad) is None
    assert bb.fp8_gemm_kernel_name(0, 64, 64) == "none"
    assert bb.fp8_gemm_gated_quantize_kernel_name(0, 64, 64) == "none"
    with pytest.raises(ValueError):
        bb.fp8_gemm_kernel_name(4, 64, 31)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, E4M3, "bf16", 1])
def test_kernel_name_refuses_other_types(dtype):
    for gated in (False, True):
        with pytest.raises(ValueError, match="dtype must be"):
            bb.fp8_gemm_kernel_name(4, 64, 64, dtype, gated)
    assert bb.fp8_gemm_kernel_name(4, 64, 64) == bb.fp8_gemm_kernel_name(4, 64, 64, torch.float32)


def test_queries_refuse_what_the_calls_refuse():
    """Sizes that only one of the calls refuses: 2^31 blocks of codes, more alternatives than logits
    or than 2^31 in all."""
    m, f, k = 1 << 16, 1 << 22, 32
    assert gated_quantize(m=m, n=f, k=k) == SHAPE
    assert bb.lib().fp8_gemm_gated_quantize_kernel_name(m, f, k) is None
    assert bb.lib().fp8_gemm_gated_quantize_bytes(m, f, k) == 0
    with pytest.raises(ValueError, match="invalid sizes"):
        bb.fp8_gemm_gated_quantize_kernel_name(m, f, k)
    assert bb.fp8_gemm_gated_quantize_kernel_name(m - 1, f, k) != "none"
    for rows, vocab, topk in ((1, 131072, 65), (1, 40, 41), (1 << 26, 8192, 32)):
        assert logprobs(rows=rows, vocab=vocab, ldl=vocab, topk=topk) == SHAPE
        assert bb.lib().token_logprobs_bytes(rows, vocab, topk) == 0


def test_every_kernel_has_a_tested_shape():
    """The shapes of the GPU tests reach every kernel in every form."""
    from test_gpu_fp8 import GATED, GATED_ODD, LONG, SHAPES
    half = torch.bfloat16
    name = bb.fp8_gemm_kernel_name
    largest, pair = "tile 256x256", "tile 128x128 pair"
    small = {"stream", pair, "tile 64x128", "tile 64x64"}
    assert small | {largest, "tile 128x128"} <= {name(*s, half) for s in SHAPES}
    assert {t + " over parts of K" for t in (largest, "tile 128x128", "tile 64x128", "tile 64x64")} <= {
        name(*s, half) for s in SHAPES + LONG}
    assert {t + " over parts of K" for t in (pair, "tile 64x128", "tile 64x64")} <= {
        name(*s) for s in SHAPES + LONG}
    assert any(name(*s, half).startswith(largest + ", then") for s in SHAPES)
    assert small <= {name(*s) for s in SHAPES}
    assert any(name(*s).startswith(pair + ", then") for s in SHAPES)
    gated = GATED + GATED_ODD
    assert small | {largest, "tile 128x128"} <= {name(*s, half, gated=True) for s in gated}
    assert any(name(*s, half, gated=True).startswith(largest + ", then") for s in gated)
    assert small <= {name(*s, gated=True) for s in gated}
    codes = {(bb.fp8_gemm_gated_quantize_kernel_name(*s),
              bb.lib().fp8_gemm_gated_quantize_bytes(*s) > 0) for s in GATED}
    assert {("stream", True), ("tile 64x64", True), ("tile 64x128", True), ("tile 64x256", False),
            (largest, False), (largest + ", then tile 64x256", False)} <= codes


def test_few_rows_of_many_columns():
    """Few rows stream their weights unless the workgroups' beginnings and ends are what counts:
    many columns of a short K, or so many that more than four rows are better off in tiles."""
    half, name = torch.bfloat16, bb.fp8_gemm_kernel_name
    for dt in (half, None):
        for m, n, k in ((1, 5120, 5120), (16, 8192, 160), (16, 17408, 5120), (16, 49152, 5120),
                        (1, 131072, 5120), (4, 262144, 5120), (32, 8192, 5120)):
            assert name(m, n, k, dt) == "stream", (m, n, k, dt)
        for m, n, k in ((1, 17408, 160), (16, 131072, 5120), (5, 65536, 5120), (16, 131072, 160),
                        (32, 17408, 5120)):
            assert name(m, n, k, dt).startswith("tile"), (m, n, k, dt)
        assert name(16, 17408, 1024, dt, gated=True) == "stream"
    assert name(16, 17408, 1024, half).startswith("tile") and name(16, 17408, 1024) == "stream"
    assert bb.fp8_gemm_gated_quantize_kernel_name(16, 17408, 160) == "stream"


def test_every_pair_of_kernels_and_every_gated_kernel_over_long_k_has_a_tested_shape():
    from test_gpu_fp8 import (GATED, GATED_LONG, GATED_ODD, GATED_SIDE_BY_SIDE, SHAPES,
                              SIDE_BY_SIDE)
    half = torch.bfloat16
    name, codes = bb.fp8_gemm_kernel_name, bb.fp8_gemm_gated_quantize_kernel_name
    largest, pair = "tile 256x256", "tile 128x128 pair"
    rest = {"tile 128x128", "tile 64x128", "tile 64x64"}
    behind = {largest + ", then " + t for t in rest | {pair}}
    behind_pair = {pair + ", then " + t for t in ("tile 64x128", "tile 64x64")}
    assert behind <= {name(*s, half) for s in SHAPES + SIDE_BY_SIDE}
    assert behind_pair <= {name(*s) for s in SHAPES + SIDE_BY_SIDE}
    gated = GATED + GATED_ODD + GATED_SIDE_BY_SIDE
    assert behind <= {name(*s, half, gated=True) for s in gated}
    assert behind_pair <= {name(*s, gated=True) for s in gated}
    small = {"stream", pair, "tile 64x128", "tile 64x64"}
    assert small | rest | {largest} <= {name(*s, half, gated=True) for s in GATED_LONG}
    assert small | behind_pair <= {name(*s, gated=True) for s in GATED_LONG}
    assert {"stream", largest, "tile 64x128", "tile 64x64", "tile 64x256",
            largest + ", then tile 64x256"} <= {codes(*s) for s in GATED_LONG if s[1] % 32 == 0}


# ------------------------------------------------------------------ binding

def codes_of(m, k):
    return torch.zeros(m, k).to(E4M3)


def weights(n=70, k=160):
    return bb.Fp8Weights(codes_of(n, k), torch.ones((n + 127) // 128, (k + 127) // 128))


def refused(match, call, *args, **kwargs):
    with pytest.raises(ValueError, match=match):
        call(*args, **kwargs)


def test_quantize_binding_refusals():
    q = bb.quantize_fp8
    x = torch.zeros(4, 160)
    refused("2-D", q, torch.zeros(4))
    refused("2-D", q, None)
    refused("dtype", q, x.half())
    refused("multiple of 32", q, torch.zeros(4, 100))
    refused("multiple of 32", q, torch.zeros(4, 0))
    refused("unit column stride", q, torch.zeros(160, 4).t())
    refused("row stride", q, torch.zeros(1, 160).expand(4, 160))
    refused("block_rows", q, x, block_rows=32)
    refused("dtype", q, x, codes=torch.zeros(4, 160))
    refused("shape", q, x, codes=codes_of(4, 128))
    refused("contiguous", q, x, codes=codes_of(4, 320)[:, ::2])
    refused("shape", q, x, scales=torch.zeros(4, 1))
    refused("shape", q, x, block_rows=128, scales=torch.zeros(4, 2))
    refused("cuda device", q, x)
    refused("cuda device", bb.quantize_weights_fp8, x)
    big = torch.zeros(4 * 160 + 16)
    x = big[:640].view(4, 160)
    refused("codes overlaps x", q, x, codes=big.view(E4M3)[:640].view(4, 160))
    refused("scales overlaps x", q, x, scales=big[632:640].view(4, 2))
    both = torch.zeros(160)
    refused("scales overlaps codes", q, x, codes=both.view(E4M3).view(4, 160),
            scales=both[:8].view(4, 2))


def test_product_binding_refusals():
    f = bb.fp8_gemm
    c, s, w = codes_of(4, 160), torch.ones(4, 2), weights()
    refused("2-D", f, None, s, w)
    refused("2-D", f, c, s[0], w)
    refused("codes has dtype", f, c.float(), s, w)
    refused("codes has dtype", f, c.view(torch.uint8), s, w)
    refused("codes has shape", f, codes_of(4, 128), s, w)
    refused("contiguous", f, codes_of(4, 320)[:, :160], s, w)
    refused("scales has dtype", f, c, s.double(), w)
    refused("scales has shape", f, c, torch.ones(4, 5), w)
    refused("scales must be contiguous", f, c, torch.ones(2, 4).t(), w)
    refused("weights' codes has dtype", f, c, s, bb.Fp8Weights(w.codes.float(), w.scales))
    refused("weights' scales has shape", f, c, s, bb.Fp8Weights(w.codes, torch.ones(70, 2)))
    refused("weights have no rows", f, c, s, bb.Fp8Weights(codes_of(0, 160), torch.ones(0, 2)))
    refused("multiple of 32", f, codes_of(4, 40), torch.ones(4, 1), weights(8, 40))
    refused("y has dtype", f, c, s, w, dtype=torch.float16)
    refused("dtype must be", f, c, s, w, dtype="bf16")
    refused("y has dtype", f, c, s, w, y=torch.zeros(4, 70), dtype=torch.bfloat16)
    refused("y has shape", f, c, s, w, y=torch.zeros(4, 71))
    refused("row stride", f, c, s, w, y=torch.zeros(1, 70).expand(4, 70))
    refused("unit column stride", f, c, s, w, y=torch.zeros(70, 4).t())
    refused("cuda device", f, c, s, w)
    buf = torch.zeros(4 * 70)
    refused("y overlaps codes", f, buf.view(E4M3)[:640].view(4, 160), s, w, y=buf.view(4, 70))
    refused("y overlaps scales", f, c, buf[:8].view(4, 2), w, y=buf.view(4, 70))
    refused("y overlaps the weights' scales", f, c, s, bb.Fp8Weights(w.codes, buf[:2].view(1, 2)),
            y=buf.view(4, 70))


def test_gated_binding_refusals():
    c, s = codes_of(4, 160), torch.ones(4, 2)
    g, u = weights(96), weights(96)
    for f in (bb.fp8_gemm_gated, bb.fp8_gemm_gated_quantize):
        refused("activation must be", f, c, s, g, u, activation="swish")
        refused("activation must be", f, c, s, g, u, activation=None)
        refused("up projection's codes has shape", f, c, s, g, weights(64))
        refused("up projection's scales has shape", f, c, s, g,
                bb.Fp8Weights(u.codes, torch.ones(2, 2)))
        refused("gate's codes has dtype", f, c, s, bb.Fp8Weights(g.codes.float(), g.scales), u)
        refused("cuda device", f, c, s, g, u)
    refused("y has shape", bb.fp8_gemm_gated, c, s, g, u, y=torch.zeros(4, 95))
    q = bb.fp8_gemm_gated_quantize
    refused("F = 70 is not a multiple of 32", q, c, s, weights(70), weights(70))
    refused("out_codes has shape", q, c, s, g, u, out_codes=codes_of(4, 64))
    refused("out_codes has dtype", q, c, s, g, u, out_codes=torch.zeros(4, 96))
    refused("out_scales has shape", q, c, s, g, u, out_scales=torch.zeros(4, 2))
    refused("out_codes overlaps codes", q, c, s, g, u, out_codes=c.view(-1)[:384].view(4, 96))
    refused("out_scales overlaps scales", q, c, s, g, u, out_scales=s.view(-1)[:4].view(4, 1))


def test_logprobs_binding_refusals():
    f = bb.token_logprobs
    x, t = torch.zeros(4, 50), torch.zeros(4, dtype=torch.int64)
    refused("2-D", f, x[0])
    refused("dtype", f, x.half())
    refused("no columns", f, torch.zeros(4, 0))
    refused("unit column stride", f, torch.zeros(50, 4).t())
    refused("row stride", f, torch.zeros(1, 50).expand(4, 50))
    refused("tokens has dtype", f, x, t.float())
    refused("tokens has shape", f, x, t[:3])
    refused("tokens has shape", f, x, t.view(4, 1))
    refused("tokens must be contiguous", f, x, torch.zeros(8, dtype=torch.int64)[::2])
    refused("topk must be", f, x, t, topk=65)
    refused("topk must be", f, x, t, topk=-1)
    refused("topk must be", f, torch.zeros(4, 3), t, topk=4)
    refused("logprobs needs tokens", f, x, logprobs=torch.zeros(4))
    refused("logprobs has shape", f, x, t, logprobs=torch.zeros(3))
    refused("entropy has dtype", f, x, t, entropy=torch.zeros(4).double())
    refused("ids has dtype", f, x, t, topk=2, ids=torch.zeros(4, 2, dtype=torch.int64))
    refused("top has shape", f, x, t, topk=2, top=torch.zeros(4, 3))
    refused("cuda device", f, x, t)
    refused("entropy overlaps logits", f, x, t, entropy=x[0, :4])
    refused("logprobs overlaps tokens", f, x, t, logprobs=t.view(torch.float32)[:4])
    e = torch.zeros(8)
    refused("entropy overlaps logprobs", f, x, t, logprobs=e[:4], entropy=e[2:6])
    refused("top overlaps ids", f, x, t, topk=2, ids=e.view(torch.int32).view(4, 2),
            top=e.view(4, 2))
    with pytest.raises(TypeError):
        f(x, t, topk="five")

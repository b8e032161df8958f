"""Refusals of the operators between the products (norm and quantize, decode,
product epilogue, routing): the C ABI reports every argument error from the
host before any HIP call, and the binding checks every tensor first.  Pointers
of the ABI tests are never dereferenced.
"""
import ctypes
import random

import pytest
import torch

from bit_prefill_gemm_amd import binding as bb

OK, NULL, SHAPE, ALIGN, DTYPE, STAMP, DEVICE = 0, 1, 2, 3, 4, 5, 7
P = ctypes.c_void_p(0x100000)
MIS = ctypes.c_void_p(0x100004)
ODD = ctypes.c_void_p(0x100001)
NUL = ctypes.c_void_p(0)
INF, NAN = float("inf"), float("nan")

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls would run")


# ------------------------------------------------------------------ C ABI

def norm(x=P, x_dt=0, ldx=128, r=P, r_dt=0, ldr=128, h=P, ldh=128, w=P, w_dt=0, eps=1e-6, m=4,
         k=128, bits=4, rot=32, codes=P, scales=P):
    return bb.lib().rmsnorm_quantize_act(x, x_dt, ldx, r, r_dt, ldr, h, ldh, w, w_dt, eps, m, k,
                                         bits, rot, codes, scales, NUL)


@pytest.mark.parametrize("args,status", [
    (dict(x_dt=2), DTYPE), (dict(r_dt=-1), DTYPE), (dict(w_dt=7), DTYPE), (dict(bits=5), DTYPE),
    (dict(rot=16), SHAPE), (dict(m=-1), SHAPE), (dict(m=1 << 31), SHAPE), (dict(k=0), SHAPE),
    (dict(k=48, ldx=64), SHAPE), (dict(k=96, rot=64), SHAPE), (dict(k=192, rot=128), SHAPE),
    (dict(k=65568, ldx=65568, ldr=65568, ldh=65568), SHAPE), (dict(ldx=127), SHAPE),
    (dict(ldr=100), SHAPE), (dict(ldh=100), SHAPE), (dict(eps=0.0), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=INF), SHAPE), (dict(eps=NAN), SHAPE),
    (dict(x=NUL), NULL), (dict(codes=NUL), NULL), (dict(scales=NUL), NULL),
    (dict(x=MIS), ALIGN), (dict(r=MIS), ALIGN), (dict(h=MIS), ALIGN), (dict(w=MIS), ALIGN),
    (dict(codes=MIS), ALIGN), (dict(scales=MIS), ALIGN), (dict(ldx=130), ALIGN),
    (dict(ldr=130), ALIGN), (dict(ldh=130), ALIGN),
])
def test_norm_abi_refusals(args, status):
    assert norm(**args) == status


@no_gpu
@pytest.mark.parametrize("args", [
    {}, dict(r=NUL, r_dt=9, ldr=-5, h=MIS, ldh=3),  # without a residual its arguments are not used
    dict(h=NUL, ldh=1), dict(w=NUL, w_dt=9), dict(m=0, x=NUL, codes=NUL, scales=NUL),
    dict(rot=0), dict(rot=128, bits=8), dict(k=65536, ldx=65536, ldr=65536, ldh=65536),
])
def test_norm_abi_valid_calls_reach_the_device_check(args):
    assert norm(**args) == DEVICE


def decode(codes=P, scales=P, bits=4, rot=32, m=4, k=128, y=P, y_dt=0, ldy=128):
    return bb.lib().dequantize_act(codes, scales, bits, rot, m, k, y, y_dt, ldy, NUL)


@pytest.mark.parametrize("args,status", [
    (dict(y_dt=3), DTYPE), (dict(bits=3), DTYPE), (dict(rot=33), SHAPE), (dict(m=-2), SHAPE),
    (dict(k=16), SHAPE), (dict(k=96, rot=128), SHAPE), (dict(ldy=96), SHAPE),
    (dict(codes=NUL), NULL), (dict(scales=NUL), NULL), (dict(y=NUL), NULL),
    (dict(codes=MIS), ALIGN), (dict(scales=MIS), ALIGN), (dict(y=MIS), ALIGN),
    (dict(ldy=130), ALIGN),
])
def test_decode_abi_refusals(args, status):
    assert decode(**args) == status


def desc(n=64, k=128, rotation=32, e=1):
    return bb.WeightsDesc(0x57475042, 1, rotation, 3, n, k, e,
                          e * (n // 32) * ((k // 32 + 3) // 4) * 2304, 2048)


def product(codes=P, scales=P, bits=4, rot=32, m=4, w=None, image=P, y=P, y_dt=0, ldy=64,
            no_ep=False, **ep):
    ep = bb.Epilogue(**{**dict(bias=0x100000, residual=0x100000, ldr=64), **ep})
    w = desc() if w is None else w
    return bb.lib().w4a4_gemm_epilogue(codes, scales, bits, rot, m, ctypes.byref(w), image,
                                       None if no_ep else ctypes.byref(ep), y, y_dt, ldy, NUL)


@pytest.mark.parametrize("args,status", [
    (dict(no_ep=True), NULL), (dict(y_dt=2), DTYPE), (dict(bias_dt=2), DTYPE),
    (dict(residual_dt=5), DTYPE), (dict(act=-1), DTYPE), (dict(act=5), DTYPE),
    (dict(bits=6), DTYPE), (dict(rot=1), SHAPE), (dict(rot=0), STAMP), (dict(rot=64), STAMP),
    (dict(w=desc(e=2)), STAMP), (dict(m=-1), SHAPE), (dict(ldr=63), SHAPE), (dict(ldy=32), SHAPE),
    (dict(bias=0x100002), ALIGN), (dict(bias=0x100001, bias_dt=1), ALIGN),
    (dict(residual=0x100002), ALIGN), (dict(residual=0x100001, residual_dt=1), ALIGN),
    (dict(codes=NUL), NULL), (dict(image=NUL), NULL), (dict(y=NUL), NULL), (dict(y=MIS), ALIGN),
    (dict(ldy=66), ALIGN), (dict(ldy=68, y_dt=1), ALIGN),
])
def test_product_abi_refusals(args, status):
    assert product(**args) == status


@no_gpu
@pytest.mark.parametrize("args", [
    {}, dict(bias=0, bias_dt=9, residual=0, residual_dt=9, ldr=-1), dict(ldr=65, residual=0x100004),
    dict(residual=0x100002, residual_dt=1, bias=0x100002, bias_dt=1),
    dict(rot=0, w=desc(rotation=0)), dict(rot=128, w=desc(rotation=128)), dict(act=4, y_dt=1),
])
def test_product_abi_valid_calls_reach_the_device_check(args):
    assert product(**args) == DEVICE


def route(logits=P, dt=0, tokens=4, experts=64, ldl=64, score=0, bias=P, groups=8, kept=4, gs=1,
          topk=8, renorm=1, scale=1.0, ids=P, weights=P):
    return bb.lib().moe_route_topk(logits, dt, tokens, experts, ldl, score, bias, groups, kept, gs,
                                   topk, renorm, scale, ids, weights, NUL)


@pytest.mark.parametrize("args,status", [
    (dict(dt=2), DTYPE), (dict(score=2), DTYPE), (dict(gs=2), DTYPE), (dict(tokens=-1), SHAPE),
    (dict(experts=0), SHAPE), (dict(experts=520, ldl=520), SHAPE), (dict(ldl=63), SHAPE),
    (dict(groups=0), SHAPE), (dict(groups=7), SHAPE), (dict(groups=64), SHAPE),
    (dict(experts=260, ldl=260, groups=65), SHAPE), (dict(kept=0), SHAPE), (dict(kept=9), SHAPE),
    (dict(topk=0), SHAPE), (dict(topk=33), SHAPE), (dict(groups=1, kept=1, topk=65), SHAPE),
    (dict(experts=512, ldl=512, groups=1, kept=1, topk=65), SHAPE),
    (dict(tokens=(1 << 17) + 1), SHAPE), (dict(scale=INF), SHAPE), (dict(scale=NAN), SHAPE),
    (dict(logits=NUL), NULL), (dict(ids=NUL), NULL), (dict(weights=NUL), NULL),
    (dict(logits=ODD), ALIGN), (dict(logits=ODD, dt=1), ALIGN), (dict(bias=ODD), ALIGN),
    (dict(ids=ODD), ALIGN), (dict(weights=ODD), ALIGN),
    (dict(logits=ctypes.c_void_p(0x100002)), ALIGN),
])
def test_route_abi_refusals(args, status):
    assert route(**args) == status


@no_gpu
@pytest.mark.parametrize("args", [
    {}, dict(groups=64, kept=64, gs=0, topk=64), dict(tokens=0, logits=NUL, ids=NUL, weights=NUL),
    dict(tokens=1 << 17), dict(bias=NUL), dict(logits=ctypes.c_void_p(0x100002), dt=1, ldl=65),
    dict(groups=1, kept=1, experts=1, topk=1), dict(scale=-2.5),
])
def test_route_abi_valid_calls_reach_the_device_check(args):
    assert route(**args) == DEVICE


# ------------------------------------------------------------------ binding

def raises(fn, *args, match, **kwargs):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kwargs)


def test_norm_binding_checks():
    f = bb.rmsnorm_quantize_act
    x = torch.zeros(4, 128)
    raises(f, [1.0], match="x must be a 2-D tensor")
    raises(f, x[0], match="x must be a 2-D tensor")
    raises(f, x.half(), match="x has dtype")
    raises(f, torch.zeros(128, 4).t(), match="unit column stride")
    raises(f, torch.zeros(1, 128).expand(4, 128), match="unit column stride")
    raises(f, x, act_bits=6, match="act_bits")
    raises(f, x, rotation=16, match="rotation must be")
    raises(f, torch.zeros(4, 96), rotation=64, match="K = 96 is not")
    raises(f, torch.zeros(4, 0), match="K = 0 is not")
    raises(f, x, residual=torch.zeros(3, 128), match="residual has shape")
    raises(f, x, residual=x.double(), match="residual has dtype")
    raises(f, x, h=x, match="h needs a residual")
    raises(f, x, residual=x, h=x.bfloat16(), match="h has dtype")
    raises(f, x, residual=x, h=torch.zeros(4, 64), match="h has shape")
    raises(f, x, weight=torch.zeros(64), match="weight has shape")
    raises(f, x, weight=torch.zeros(128).half(), match="weight has dtype")
    raises(f, x, weight=torch.zeros(256)[::2], match="weight must be contiguous")
    raises(f, x, weight=3.0, match="weight must be a torch tensor")
    raises(f, x, codes=torch.zeros(4, 128, dtype=torch.uint8), match="codes has shape")
    raises(f, x, scales=torch.zeros(4, 3), match="scales has shape")
    raises(f, x, residual=x.bfloat16(), weight=x[0].clone(), match="cuda device")


def test_decode_binding_checks():
    f = bb.dequantize_act
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4)
    raises(f, codes, None, match="scales must be a 2-D tensor")
    raises(f, codes, scales, 8, match="codes has shape")
    raises(f, codes, scales, rotation=8, match="rotation must be")
    raises(f, codes[:, :48].contiguous(), scales[:, :3].contiguous(), rotation=128, match="K = 96")
    raises(f, codes, scales, y=torch.zeros(4, 64), match="y has shape")
    raises(f, codes, scales, y=torch.zeros(4, 128), dtype=torch.bfloat16, match="y has dtype")
    raises(f, codes, scales, dtype=torch.float16, match="y has dtype")
    raises(f, codes, scales, match="cuda device")


def test_product_binding_checks():
    f = bb.w4a4_gemm_epilogue
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4)
    w = bb.Weights(desc(), torch.zeros(desc().bytes, dtype=torch.uint8))
    raises(f, codes, scales, 3, w, match="act_bits")
    raises(f, codes[0], scales, 4, w, match="codes must be a 2-D tensor")
    raises(f, codes, scales, 4, w, activation="tanh", match="activation must be")
    raises(f, codes, scales, 4, w, bias=torch.zeros(63), match="bias has shape")
    raises(f, codes, scales, 4, w, bias=torch.zeros(64).half(), match="bias has dtype")
    raises(f, codes, scales, 4, w, bias=torch.zeros(128)[::2], match="bias must be contiguous")
    raises(f, codes, scales, 4, w, bias=1.0, match="bias must be a torch tensor")
    raises(f, codes, scales, 4, w, residual=torch.zeros(4, 63), match="residual has shape")
    raises(f, codes, scales, 4, w, residual=torch.zeros(64), match="residual must be a 2-D")
    raises(f, codes, scales, 4, w, residual=torch.zeros(1, 64).expand(4, 64), match="unit column")
    raises(f, codes, scales, 4, w, y=torch.zeros(4, 64).half(), match="y has dtype")
    raises(f, codes, scales, 4, w, y=torch.zeros(4, 64), dtype=torch.bfloat16, match="y has dtype")
    raises(f, codes, scales, 4, w, y=7, match="y must be a torch tensor")
    raises(f, codes, scales, 4, w, y=torch.zeros(3, 64), match="y has shape")
    raises(f, codes, scales, 4, w, bias=torch.zeros(64), residual=torch.zeros(4, 64).bfloat16(),
           dtype=torch.bfloat16, match="cuda device")


@pytest.mark.parametrize("rotation", [16, -32, 256, (1 << 32) + 32, 1 << 32])
def test_product_binding_refuses_other_spans(rotation):
    """Also those that a C int would turn into a valid one."""
    W = bb.Weights(desc(n=96), torch.zeros(3 * 2304, dtype=torch.uint8))
    raises(bb.w4a4_gemm_epilogue, torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4), 4, W,
           rotation=rotation, match="rotation must be")


@pytest.mark.parametrize("bits,m,n,k,name", [
    (4, 0, 5120, 5120, "none"), (4, 1, 1024, 5120, "weight-stream chunks"),
    (4, 1, 5120, 5120, "weight-stream"), (8, 77, 1056, 2080, "weight-stream chunks"),
    (4, 512, 5120, 5120, "wide 64x160"), (8, 512, 5120, 17408, "tiled 64x160"),
    (4, 1024, 17408, 5120, "strip 32x128"), (8, 1024, 17376, 5120, "strip 32x128"),
    (4, 1024, 1056, 2080, "tiled 64x32"),
])
def test_product_epilogue_kernels(bits, m, n, k, name):
    if m == 0:
        name = bb.lib().w4a4_gemm_kernel_name(bits, 0, ctypes.byref(desc(n, k))).decode()
    got = bb.lib().w4a4_gemm_epilogue_kernel_name(bits, m, ctypes.byref(desc(n, k)))
    assert got.decode() == name


def test_route_binding_checks():
    f = bb.moe_route_topk
    logits = torch.zeros(4, 16)
    raises(f, logits[0], 2, match="logits must be a 2-D tensor")
    raises(f, logits.double(), 2, match="logits has dtype")
    raises(f, torch.zeros(16, 4).t(), 2, match="unit column stride")
    raises(f, logits, 2, score="relu", match="score must be")
    raises(f, logits, 2, group_score="sum", match="group_score must be")
    raises(f, logits, 0, match="topk must be positive")
    raises(f, logits, 2, bias=torch.zeros(15), match="bias has shape")
    raises(f, logits, 2, bias=torch.zeros(16).bfloat16(), match="bias has dtype")
    raises(f, logits, 2, expert_of=torch.zeros(8), match="expert_of has dtype")
    raises(f, logits, 2, weights=torch.zeros(9), match="weights has shape")
    raises(f, logits.bfloat16(), 2, bias=torch.zeros(16), match="cuda device")


# ------------------------------------------------------------------ outputs over inputs

def columns(rows, *widths, dtype=torch.float32):
    """Matrices beside one another in the rows of one buffer."""
    buf = torch.zeros(rows, sum(widths), dtype=dtype)
    return buf.split(list(widths), 1)


def test_norm_binding_refuses_overlaps():
    f = bb.rmsnorm_quantize_act
    x, r = torch.zeros(4, 128), torch.zeros(5, 128)
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4)
    raises(f, x, residual=r[1:], h=r[:4], match="h overlaps the residual")
    raises(f, x, residual=r[:4], h=r[1:], match="h overlaps the residual")
    raises(f, x, residual=torch.zeros(4, 128), h=x, match="h overlaps x")
    raises(f, x, residual=x, h=x, match="h overlaps x")
    # the same memory as rows of another stride
    raises(f, x, residual=r.view(-1)[:512].view(4, 128), h=r.view(-1).as_strided((4, 128), (132, 1)),
           match="h overlaps the residual")
    raises(f, x, scales=x.view(-1)[:16].view(4, 4), match="scales overlaps x")
    raises(f, x, codes=x.view(torch.uint8).view(-1)[-256:].view(4, 64), match="codes overlaps x")
    raises(f, x, codes=codes, scales=codes.view(torch.float32).view(-1)[:16].view(4, 4),
           match="scales overlaps codes")
    w = torch.zeros(128)
    raises(f, x, weight=w, scales=w[112:].view(4, 4), match="scales overlaps the weight")
    h = torch.zeros(4, 128)
    raises(f, x, residual=r[:4], h=h, codes=h.view(torch.uint8).view(-1)[:256].view(4, 64), match="codes overlaps h")
    # no overlap: the stream where it is, a row that ends where the next matrix begins, columns of one buffer
    raises(f, x, residual=r[:4], h=r[:4], match="cuda device")
    raises(f, x[:1], residual=r[:1], h=r[:1].as_strided((1, 128), (500, 1)), match="cuda device")
    both = torch.zeros(8, 128)
    raises(f, x, residual=both[:4], h=both[4:], match="cuda device")
    a, b, c = columns(4, 128, 128, 128)
    raises(f, a, residual=b, h=c, match="cuda device")
    raises(f, a, residual=b, h=b, match="cuda device")
    raises(f, a[:1], residual=b[1:2], h=c[:1], match="cuda device")
    raises(f, c[1:2], residual=a[3:], h=b[:1], match="cuda device")
    raises(f, x, residual=r[:4], h=h, codes=codes, scales=scales, match="cuda device")
    # rows of another stride between those of the buffer's first columns
    wide = torch.zeros(8, 256)
    raises(f, x, residual=wide[:4, :128], h=wide.view(-1).as_strided((4, 128), (512, 1), 128), match="cuda device")
    raises(f, x, residual=wide[:4, :128], h=wide.view(-1).as_strided((4, 128), (388, 1), 128), match="h overlaps the residual")


def test_decode_binding_refuses_overlaps():
    f = bb.dequantize_act
    buf = torch.zeros(4 * 128 + 16)
    scales = buf[:16].view(4, 4)
    codes = torch.zeros(4, 64, dtype=torch.uint8)
    raises(f, codes, scales, y=buf[4:516].view(4, 128), match="y overlaps scales")
    raises(f, buf[-64:].view(torch.uint8).view(4, 64), scales, y=buf[16:].view(4, 128), match="y overlaps codes")
    raises(f, codes, scales, y=buf[16:].view(4, 128), match="cuda device")


def test_product_binding_refuses_overlaps():
    f = bb.w4a4_gemm_epilogue
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4)
    w = bb.Weights(desc(), torch.zeros(desc().bytes, dtype=torch.uint8))
    buf = torch.zeros(5, 64)
    raises(f, codes, scales, 4, w, residual=buf[1:], y=buf[:4], match="y overlaps the residual")
    raises(f, codes, scales, 4, w, residual=buf[:4], y=buf[1:], match="y overlaps the residual")
    # the same place, but as another type or with rows another stride apart
    raises(f, codes, scales, 4, w, residual=buf[:4].view(torch.bfloat16)[:, :64], y=buf[:4],
           match="y overlaps the residual")
    raises(f, codes, scales, 4, w, residual=buf[:4], y=buf.view(-1).as_strided((4, 64), (68, 1)),
           match="y overlaps the residual")
    raises(f, codes, scales, 4, w, bias=buf[3], y=buf[:4], match="y overlaps the bias")
    raises(f, codes, buf.view(-1)[:16].view(4, 4), 4, w, y=buf[:4], match="y overlaps scales")
    raises(f, buf.view(torch.uint8).view(-1)[:256].view(4, 64), scales, 4, w, y=buf[:4], match="y overlaps codes")
    raises(f, codes, scales, 4, w, y=w.image[:1024].view(torch.float32).view(4, 64), match="y overlaps the weight image")
    raises(f, codes, scales, 4, w, residual=buf[:4], y=buf[:4], match="cuda device")
    a, b = columns(4, 64, 64)
    raises(f, codes, scales, 4, w, residual=a, y=b, bias=buf[4], match="cuda device")
    raises(f, codes, scales, 4, w, residual=b, y=a, match="cuda device")
    a, b = columns(4, 64, 64, dtype=torch.bfloat16)
    raises(f, codes, scales, 4, w, residual=b, y=b, match="cuda device")


def test_route_binding_refuses_overlaps():
    f = bb.moe_route_topk
    buf = torch.zeros(4, 16)
    out = torch.zeros(16, dtype=torch.int32)
    raises(f, buf, 2, weights=buf.view(-1)[:8], match="weights overlaps logits")
    raises(f, buf, 2, expert_of=buf.view(torch.int32).view(-1)[56:], match="expert_of overlaps logits")
    raises(f, buf, 2, expert_of=out[:8], weights=out.view(torch.float32)[7:15], match="weights overlaps expert_of")
    b = torch.zeros(16)
    raises(f, buf, 2, bias=b, weights=b[8:], match="weights overlaps the bias")
    raises(f, buf, 2, bias=b, expert_of=out[:8], weights=out.view(torch.float32)[8:], match="cuda device")
    # columns beside the logits
    raises(f, buf[:1, :8], 2, weights=buf[0, 8:10], expert_of=out[:2], match="cuda device")


def overlap_by_bytes(a, b):
    def at(t):
        return {t.data_ptr() + i * t.stride(0) * t.element_size() + j
                for i in range(t.shape[0]) for j in range(t.shape[1] * t.element_size())}
    return bool(at(a) & at(b))


def test_overlaps_of_random_rows():
    """Against the sets of bytes: both strides, both orders, one row and many."""
    rng = random.Random(4)
    buf = torch.zeros(4096)
    met = set()
    for _ in range(600):
        m, k = rng.randint(1, 6), 32
        strides = [rng.choice([32, 36, 64, 64, 68, 96, 128]) for _ in range(2)]
        at = [4 * rng.randrange(0, 100) for _ in range(2)]
        r, h = (buf.as_strided((m, k), (s, 1), o) for s, o in zip(strides, at))
        same = at[0] == at[1] and (m == 1 or strides[0] == strides[1])
        bad = not same and overlap_by_bytes(r, h)
        met.add((bad, m == 1, strides[0] == strides[1]))
        raises(bb.rmsnorm_quantize_act, torch.zeros(m, k), residual=r, h=h,
               match="h overlaps the residual" if bad else "cuda device")
    assert len(met) == 8

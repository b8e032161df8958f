"""The 8-bit floating-point route: codes, products, the gated products, and a
feed-forward block of them.

Bars:
- codes and scales are equal bit for bit to a plain evaluation of the
  definition in fp32 steps, and lie within half a step of e4m3 of x / d;
- products of small whole codes under power-of-two scales are exact in every
  kernel: the results equal the whole-number ones bit for bit;
- products of ordinary codes lie within the rounding bounds derived below.
"""
import math
import threading

import numpy as np
import pytest

from bit_prefill_gemm_amd import binding as bb

from gpu_util import torch_mod

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of fp32


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    return t


def blocks(k):
    return (k + 127) // 128


def generator(torch, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ quantize

def plain_codes(torch, x, rows):
    """(codes, scales) of a cpu fp32 matrix, step by step."""
    m, k = x.shape
    t, b = (m + rows - 1) // rows, blocks(k)
    v = torch.zeros(t * rows, b * 128)
    v[:m, :k] = x
    v = v.view(t, rows, b, 128)
    amax = v.abs().amax((1, 3), keepdim=True)
    d = amax / torch.full_like(amax, 448.0)
    r = torch.where(d > 0, torch.minimum(1.0 / d, torch.tensor(torch.finfo(torch.float32).max)), 0.0)
    q = (v * r).to(torch.float8_e4m3fn).view(torch.uint8).view(t * rows, b * 128)[:m, :k]
    return q, d.view(t, b)


def inputs(torch, m, k, kind, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    x = torch.randn(m, k, generator=g)
    if kind == "outliers":
        x[:, torch.randperm(k, generator=g)[:max(1, k // 50)]] *= 100.0
    elif kind == "wide":  # magnitudes over the whole range of fp32, subnormal ones too
        x = torch.ldexp(x, torch.randint(-148, 119, (m, k), generator=g).float())
        x[0, :] = 0.0
        x[m // 2, k // 2:] = 0.0
    elif kind == "tiny":  # scales that underflow, or whose inverse overflows
        x = torch.ldexp(x, torch.randint(-149, -115, (m, 1), generator=g).float())
    return x


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,k,pad,kind", [
    (1, 32, 0, "normal"), (1, 5120, 0, "outliers"), (3, 96, 4, "normal"), (130, 160, 12, "wide"),
    (257, 352, 0, "outliers"), (128, 128, 4, "tiny"), (127, 2080, 36, "outliers"),
    (33, 17408, 0, "wide"), (1024, 1024, 0, "normal")])
def test_quantize(torch, m, k, pad, kind, dtype, rows):
    dt = getattr(torch, dtype)
    x = inputs(torch, m, k, kind, m * k).to(dt)
    wide = torch.full((m, k + pad), 3.0, dtype=dt, device="cuda")
    wide[:, :k] = x.cuda()
    codes, scales = bb.quantize_fp8(wide[:, :k], block_rows=rows)
    torch.cuda.synchronize()
    q, d = plain_codes(torch, x.float(), rows)
    assert torch.equal(scales.cpu().view(torch.int32), d.view(torch.int32))
    got = codes.cpu().view(torch.uint8)
    # the zero of a value that rounds to it keeps its sign in both
    assert torch.equal(got, q), torch.nonzero(got != q)[:4]
    # the formula: x / d in 64 bits, half a step of e4m3 (2^-4 of the value, 2^-10 near zero), the
    # two roundings of r and x r; a scale below 2^-126 is itself rounded to 2^-150 at most, and its
    # inverse is held to the largest fp32
    dd = d.double().repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :k]
    v = torch.where(dd > 2.0 ** -126, x.double() / dd, 0.0)
    err = (codes.cpu().double() - v).abs()
    lim = torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 8 * U) + 4 * U * v.abs()
    assert ((err <= lim) | (dd <= 2.0 ** -126)).all()


def test_quantize_special_values(torch):
    x = torch.ones(6, 256, device="cuda")
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    x[3] = 0.0
    x[4, :128] = -0.0
    codes, scales = bb.quantize_fp8(x)
    c, s = codes.float().cpu(), scales.cpu()
    assert torch.isnan(s[1, 0]) and torch.isnan(c[1, 5]) and s[1, 1] == s[0, 0]
    assert torch.isinf(s[2, 1]) and torch.isnan(c[2, 200]) and (c[2, 128:200] == 0).all()
    assert (s[3] == 0).all() and (c[3] == 0).all() and s[4, 0] == 0
    assert (c[5] == 448).all() and (c[0] == 448).all()
    c2, s2 = bb.quantize_fp8(x, block_rows=128)
    assert torch.isnan(s2[0, 0]) and torch.isinf(s2[0, 1])


def test_quantize_empty(torch):
    codes, scales = bb.quantize_fp8(torch.zeros(0, 64, device="cuda"))
    assert codes.shape == (0, 64) and scales.shape == (0, 1)


def test_quantize_more_rows_than_a_grid_holds(torch):
    """2^29 blocks and some: 2^32 threads, over several launches."""
    m, k = (1 << 29) + 77, 32
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    near = [slice(at, at + 64) for at in (0, (1 << 28) - 32, (1 << 29) - 32, m - 64)]
    for i, s in enumerate(near):
        x[s] = inputs(torch, 64, k, "normal", i).bfloat16().cuda()
    codes, scales = bb.quantize_fp8(x)
    for s in near:
        q, d = plain_codes(torch, x[s].float().cpu(), 1)
        assert torch.equal(scales[s].cpu(), d)
        assert torch.equal(codes[s].view(torch.uint8).cpu(), q)
    assert int(torch.count_nonzero(scales)) == 64 * len(near) - 19  # the last two overlap


# ------------------------------------------------------------------ products

# every kernel and both sides of its limits; odd rows and columns, K that ends inside a block
SHAPES = [(300, 256, 8192), (260, 516, 4128), (1, 1, 32), (1, 16, 96), (1, 128, 128), (2, 300, 160), (15, 129, 352), (16, 512, 1024),
          (17, 100, 256), (31, 640, 544), (33, 257, 128), (64, 384, 2080), (65, 130, 160),
          (128, 256, 512), (130, 1061, 352), (200, 512, 1152), (257, 300, 416), (300, 1536, 288),
          (513, 257, 800), (1000, 2048, 256), (33, 5120, 5120), (1, 17408, 1024),
          (65, 4100, 160), (200, 4100, 160), (1500, 1300, 160), (1500, 1300, 2080), (2050, 4100, 160),
          (1030, 17410, 544)]


def small_codes(torch, g, m, k, top=3):
    """Whole codes up to `top` in magnitude (exact in every product and sum)."""
    return torch.randint(-top, top + 1, (m, k), generator=g, device="cuda").float().to(
        torch.float8_e4m3fn)


def power_scales(torch, g, m, k):
    return torch.ldexp(torch.ones(m, k, device="cuda"),
                       torch.randint(-2, 3, (m, k), generator=g, device="cuda").float())


def wide_values(torch, codes, scales, rows):
    n, k = codes.shape
    s = scales.double().repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return codes.double() * s


def mm64(torch, a, b):
    return torch.mm(a, b.t().contiguous())


def output(torch, m, n, dtype, how):
    """(y to give, the buffer around it)"""
    if how == "new":
        return None, None
    pad = {"padded": 8, "odd": 3}[how]
    buf = torch.full((m * (n + pad) + 8,), 7.0, dtype=dtype, device="cuda")
    start = 1 if how == "odd" else 0
    return buf[start:start + m * (n + pad)].view(m, n + pad)[:, :n], buf


def check_around(torch, y, buf, how):
    """Nothing beside the rows of y was written."""
    if buf is None:
        return
    mask = torch.ones_like(buf, dtype=torch.bool)
    m, n = y.shape
    pad = {"padded": 8, "odd": 3}[how]
    start = 1 if how == "odd" else 0
    mask[start:start + m * (n + pad)].view(m, n + pad)[:, :n] = False
    assert (buf[mask] == 7.0).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_exact(torch, m, n, k, dtype):
    """Sums of whole products below 2^24 under power-of-two scales: bit for bit."""
    dt = getattr(torch, dtype)
    g = generator(torch, m + n + k)
    c, s = small_codes(torch, g, m, k), power_scales(torch, g, m, blocks(k))
    w = bb.Fp8Weights(small_codes(torch, g, n, k), power_scales(torch, g, blocks(n), blocks(k)))
    for how in ("new", "padded", "odd"):
        y, buf = output(torch, m, n, dt, how)
        got = bb.fp8_gemm(c, s, w, y=y, dtype=dt)
        assert y is None or got is y
        ref = mm64(torch, wide_values(torch, c, s, 1), wide_values(torch, w.codes, w.scales, 128))
        assert torch.equal(got, ref.to(dt)), torch.nonzero(got != ref.to(dt))[:4]
        check_around(torch, got, buf, how)


# more blocks of K than a wave holds scales of at once (60), in one piece and in parts
LONG = [(m, n, k) for m, n in ((1, 40), (20, 136), (40, 64), (70, 1300), (130, 300), (300, 520),
                               (520, 5000), (700, 1100), (1024, 2048), (2050, 4100), (39, 1),
                               (130, 301), (259, 1034), (520, 4999))
        for k in (61 * 128, 120 * 128 + 32)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n,k", LONG)
def test_product_exact_long_k(torch, m, n, k, dtype):
    """Codes of 1, 0 and -1 under scales of 1/4 to 4: at most 15392 * 256 steps of 1/16."""
    dt = getattr(torch, dtype)
    g = generator(torch, m + n + k)
    c, s = small_codes(torch, g, m, k, 1), power_scales(torch, g, m, blocks(k))
    w = bb.Fp8Weights(small_codes(torch, g, n, k, 1), power_scales(torch, g, blocks(n), blocks(k)))
    ref = mm64(torch, wide_values(torch, c, s, 1), wide_values(torch, w.codes, w.scales, 128)).to(dt)
    for how in ("new", "odd"):
        y, buf = output(torch, m, n, dt, how)
        got = bb.fp8_gemm(c, s, w, y=y, dtype=dt)
        assert torch.equal(got, ref), torch.nonzero(got != ref)[:4]
        check_around(torch, got, buf, how)


def real_codes(torch, g, m, k, rows, outliers):
    x = torch.randn(m, k, generator=g, device="cuda")
    if outliers:
        x[:, torch.randperm(k, generator=g, device="cuda")[:max(1, k // 100)]] *= 30.0
    return bb.quantize_fp8(x, block_rows=rows)


def eights(torch, a):
    """The largest magnitude of every eight consecutive k."""
    m, k = a.shape
    return a.abs().view(m, k // 8, 8)


def product_bound(torch, a, b, exact):
    """|y - exact| before the rounding to y's type.  The blocks' sums and their total: a product
    passes at most 128 + blocks additions, and its block's one multiplication by the rounded product
    of two scales; the matrix instruction may cut where fp32 rounds, so 2^-23 each.  The 8-bit
    instruction drops from each of eight products less than 2^-12 of the largest of the eight: 8
    2^-12 of that (its bound over all pairs of rows: the product of the two largest magnitudes)."""
    k = a.shape[1]
    lim = (128 + blocks(k) + 8) * 2.0 ** -23 * mm64(torch, a.abs(), b.abs())
    if not exact:
        lim = lim + 2.0 ** -9 * mm64(torch, eights(torch, a).amax(2), eights(torch, b).amax(2))
    return lim


HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}


@pytest.mark.parametrize("outliers", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(torch, m, n, k, dtype, outliers):
    dt = getattr(torch, dtype)
    g = generator(torch, m * 3 + n + k)
    c, s = real_codes(torch, g, m, k, 1, outliers)
    w = bb.Fp8Weights(*real_codes(torch, g, n, k, 128, False))
    y = bb.fp8_gemm(c, s, w, dtype=dt)
    a, b = wide_values(torch, c, s, 1), wide_values(torch, w.codes, w.scales, 128)
    ref = mm64(torch, a, b)
    lim = product_bound(torch, a, b, dtype == "float32")
    err = (y.double() - ref).abs()
    assert (err <= lim + HALF[dtype] * (ref.abs() + lim)).all(), (err / lim).max()
    # and as a whole: fp32 sums to 2^-20 of the norm; the instruction's dropped bits to 2^-12
    whole = (2.0 ** -20 if dtype == "float32" else 2.0 ** -12 + HALF[dtype]) * ref.norm()
    assert (y.double() - ref).norm() <= whole


def test_product_repeats_bit_for_bit(torch):
    g = generator(torch, 5)
    for m, n, k in ((1, 512, 2048), (70, 300, 544), (300, 520, 1024)):
        c, s = real_codes(torch, g, m, k, 1, True)
        w = bb.Fp8Weights(*real_codes(torch, g, n, k, 128, False))
        for dt in (torch.float32, torch.bfloat16):
            first = bb.fp8_gemm(c, s, w, dtype=dt)
            for _ in range(5):
                assert torch.equal(bb.fp8_gemm(c, s, w, dtype=dt), first)


def test_product_nan_stays_in_its_row_and_column(torch):
    """A NaN code or scale reaches the results of its row or columns, and no others."""
    g = generator(torch, 6)
    for m, n, k in ((3, 150, 160), (40, 260, 352), (270, 300, 288)):
        for dt in (torch.float32, torch.bfloat16):
            c, s = real_codes(torch, g, m, k, 1, False)
            w = bb.Fp8Weights(*real_codes(torch, g, n, k, 128, False))
            c.view(torch.uint8)[m - 1, k - 1] = 0x7f
            w.codes.view(torch.uint8)[n - 1, 0] = 0xff
            y = torch.isnan(bb.fp8_gemm(c, s, w, dtype=dt))
            assert y[m - 1].all() and y[:, n - 1].all() and not y[:m - 1, :n - 1].any()


def test_product_no_rows(torch):
    w = bb.Fp8Weights(*bb.quantize_fp8(torch.ones(40, 64, device="cuda"), 128))
    y = bb.fp8_gemm(*bb.quantize_fp8(torch.zeros(0, 64, device="cuda")), w)
    assert y.shape == (0, 40)
    c, s = bb.fp8_gemm_gated_quantize(*bb.quantize_fp8(torch.zeros(0, 64, device="cuda")),
                                      bb.quantize_weights_fp8(torch.ones(64, 64, device="cuda")),
                                      bb.quantize_weights_fp8(torch.ones(64, 64, device="cuda")))
    assert c.shape == (0, 64) and s.shape == (0, 1)


def test_product_offsets_past_32_bits(torch):
    """Codes, weights and outputs over 4 GiB: the last rows and columns are right."""
    k, n = 16384, 300000
    g = generator(torch, 9)
    w = bb.Fp8Weights(torch.zeros(n, k, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                      torch.ones(blocks(n), blocks(k), device="cuda"))
    tail = small_codes(torch, g, 200, k)
    w.codes.view(torch.uint8)[-200:] = tail.view(torch.uint8)
    for m in (1, 20, 200):
        c = small_codes(torch, g, m, k)
        s = torch.ones(m, blocks(k), device="cuda")
        y = bb.fp8_gemm(c, s, w, dtype=torch.bfloat16)
        ref = mm64(torch, c.double(), tail.double()).to(torch.bfloat16)
        assert torch.equal(y[:, -200:], ref) and (y[:, :-200] == 0).all()
    # rows of activations past 4 GiB, against a few columns
    small = bb.Fp8Weights(tail[:40].contiguous(), torch.ones(1, blocks(k), device="cuda"))
    y = bb.fp8_gemm(w.codes, torch.ones(n, blocks(k), device="cuda"), small, dtype=torch.bfloat16)
    ref = mm64(torch, tail.double(), tail[:40].double()).to(torch.bfloat16)
    assert torch.equal(y[-200:], ref) and (y[:-200] == 0).all()


# ------------------------------------------------------------------ gated

def act64(torch, g, act):
    if act == "relu":
        return torch.where(g > 0, g, 0.0)
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return g * torch.special.ndtr(g)
    if act == "gelu_tanh":
        return g * torch.sigmoid(2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3))
    return g


GATED = [(1, 32, 32), (1, 1024, 5120), (2, 160, 96), (16, 288, 352), (17, 96, 160), (33, 416, 512),
         (65, 128, 1024), (77, 1056, 2080), (130, 640, 416), (200, 1280, 256), (300, 992, 544),
         (513, 160, 288), (1024, 512, 256), (65, 4096, 160), (65, 5120, 1056), (200, 4096, 160),
         (200, 4096, 2080), (1030, 2048, 160), (1500, 2688, 160), (2050, 4096, 160)]

GATED_ODD = [(5, 33, 64), (100, 1061, 160), (300, 129, 96), (200, 4100, 2080), (1030, 4100, 288), (1500, 2700, 160)]


def gated_case(torch, m, f, k, seed):
    g = generator(torch, seed)
    c, s = real_codes(torch, g, m, k, 1, True)
    spread = 2.0 / np.sqrt(k)

    def weights():
        x = torch.randn(f, k, generator=g, device="cuda") * spread
        return bb.quantize_weights_fp8(x)
    return c, s, weights(), weights()


def gated_reference(torch, c, s, gate, up, act, exact):
    """(h in 64 bits, bound of the fp32 h before its rounding).  h = act(g) u: |act'| <= 1.14 for
    every activation, its evaluation within 2^-19 of |g| (gelu_tanh: the argument's error, up to
    88 roundings of 2^-24 where the sigmoid still counts), the product one rounding."""
    a = wide_values(torch, c, s, 1)
    wg, wu = (wide_values(torch, w.codes, w.scales, 128) for w in (gate, up))
    g, u = mm64(torch, a, wg), mm64(torch, a, wu)
    dg, du = product_bound(torch, a, wg, exact), product_bound(torch, a, wu, exact)
    t = act64(torch, g, act)
    lim = (1.14 * dg + 2.0 ** -19 * g.abs()) * (u.abs() + du) + t.abs() * du
    h = t * u
    return h, lim + U * (h.abs() + lim)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,f,k", GATED + GATED_ODD)
def test_gated(torch, m, f, k, dtype, act):
    dt = getattr(torch, dtype)
    c, s, gate, up = gated_case(torch, m, f, k, m + f + k)
    for how in ("new", "odd"):
        y, buf = output(torch, m, f, dt, how)
        y = bb.fp8_gemm_gated(c, s, gate, up, activation=act, y=y, dtype=dt)
        h, lim = gated_reference(torch, c, s, gate, up, act, dtype == "float32")
        err = (y.double() - h).abs()
        assert (err <= lim + HALF[dtype] * (h.abs() + lim)).all(), (err / lim).max()
        check_around(torch, y, buf, how)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("m,f,k", GATED)
def test_gated_quantize(torch, m, f, k, act):
    """Scales: the block's largest |h| / 448.  Codes: c d within half a step of e4m3 of h (2^-4 of
    the value, 2^-10 d near zero) plus h's own error; h / d is formed with three roundings, and may
    round to the other side of a step by h's error, which the bound holds as it is a value's."""
    c, s, gate, up = gated_case(torch, m, f, k, m + f + k)
    codes, scales = bb.fp8_gemm_gated_quantize(c, s, gate, up, activation=act)
    h, lim = gated_reference(torch, c, s, gate, up, act, False)
    pad = blocks(f) * 128 - f
    top = torch.nn.functional.pad(h.abs(), (0, pad)).view(m, -1, 128).amax(2)
    slack = torch.nn.functional.pad(lim, (0, pad)).view(m, -1, 128).amax(2)
    assert ((scales.double() * 448 - top).abs() <= slack + 2 * U * (top + slack)).all()
    d = scales.double().repeat_interleave(128, 1)[:, :f]
    err = (codes.double() * d - h).abs()
    size = h.abs() + lim
    step = torch.maximum(size * 2.0 ** -4, 2.0 ** -10 * d)
    assert (err <= step + lim + 4 * U * size).all(), (err / (step + lim)).max()


def test_codes_of_few_rows_are_those_of_the_fp32_values(torch):
    for m, f, k in ((1, 1024, 2080), (16, 640, 544), (30, 96, 5120)):
        g = generator(torch, m)
        c, s = real_codes(torch, g, m, k, 1, True)
        ws = [bb.Fp8Weights(*real_codes(torch, g, f, k, 128, False)) for _ in range(2)]
        want = bb.quantize_fp8(bb.fp8_gemm_gated(c, s, *ws, dtype=torch.float32))
        for a, b in zip(bb.fp8_gemm_gated_quantize(c, s, *ws), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_gated_exact_relu(torch):
    """Whole codes: every kernel's gate and up columns are where they belong, bit for bit."""
    for m, f, k in GATED + GATED_ODD:
        g = generator(torch, m + f)
        c, s = small_codes(torch, g, m, k, 1), power_scales(torch, g, m, blocks(k))

        def weights():
            return bb.Fp8Weights(small_codes(torch, g, f, k, 1),
                                 power_scales(torch, g, blocks(f), blocks(k)))
        gate, up = weights(), weights()
        a = wide_values(torch, c, s, 1)
        wg, wu = (wide_values(torch, w.codes, w.scales, 128) for w in (gate, up))
        h = torch.relu(mm64(torch, a, wg)) * mm64(torch, a, wu)
        for dt in (torch.float32, torch.bfloat16):
            # both factors are whole multiples of 2^-4 below 2^17: the fp32 product rounds once
            ref = h.float().to(dt)
            got = bb.fp8_gemm_gated(c, s, gate, up, activation="relu", dtype=dt)
            assert torch.equal(got, ref), (m, f, k, dt)
        if f % 32 == 0:
            codes, scales = bb.fp8_gemm_gated_quantize(c, s, gate, up, activation="relu")
            q, d = plain_codes(torch, h.float().cpu(), 1)
            assert torch.equal(scales.cpu(), d), (m, f, k)
            assert torch.equal(codes.cpu().view(torch.uint8) & 0x7f, q & 0x7f), (m, f, k)


# ------------------------------------------------------------------ together

def block(bb, torch, x, ws):
    """A feed-forward block as a program runs it, and a head on top of it."""
    gate, up, down, head = ws
    c, s = bb.quantize_fp8(x)
    h, hs = bb.fp8_gemm_gated_quantize(c, s, gate, up)
    y = bb.fp8_gemm(h, hs, down, dtype=torch.bfloat16)
    x = x + y
    logits = bb.fp8_gemm(*bb.quantize_fp8(x), head, dtype=torch.float32)
    return (x, logits) + bb.token_logprobs(logits, topk=4)[1:]


def block_weights(torch, k, f, v, seed):
    g = generator(torch, seed)
    make = lambda n, d: bb.quantize_weights_fp8(  # noqa: E731
        torch.randn(n, d, generator=g, device="cuda") / np.sqrt(d))
    return make(f, k), make(f, k), make(k, f), make(v, k)


@pytest.mark.parametrize("m", [1, 24, 150, 300])
def test_block_against_64_bits(torch, m):
    """The whole chain: fp64 of the unquantized steps is off by the codes' roundings (2^-4 a value,
    a third of that in the mean, over independent values), so the norm agrees to 2^-4."""
    k, f, v = 512, 1152, 1000
    ws = block_weights(torch, k, f, v, m)
    x = torch.randn(m, k, generator=generator(torch, m), device="cuda").to(torch.bfloat16)
    out, logits, entropy, ids, top = block(bb, torch, x, ws)
    a = x.double()
    wg, wu, wd, wh = (wide_values(torch, w.codes, w.scales, 128) for w in ws)
    h = act64(torch, mm64(torch, a, wg), "silu") * mm64(torch, a, wu)
    ref = a + mm64(torch, h, wd)
    assert (out.double() - ref).norm() <= 2.0 ** -4 * ref.norm()
    ref = mm64(torch, out.double(), wh)
    assert (logits.double() - ref).norm() <= 2.0 ** -4 * ref.norm()
    p = torch.log_softmax(logits.double(), 1)
    assert torch.equal(ids, torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :4].int())
    assert (top.double() - torch.gather(p, 1, ids.long())).abs().max() <= 1e-5
    assert (entropy.double() + (p.exp() * p).sum(1)).abs().max() <= 1e-4


@pytest.mark.parametrize("m", [1, 40, 300])
def test_block_from_graphs(torch, m):
    """Two captured graphs of the chain, replayed several times with eager work between."""
    ws = block_weights(torch, 256, 640, 777, 3)
    xs = [torch.randn(m, 256, generator=generator(torch, i), device="cuda") for i in range(2)]
    ins, outs, graphs = [x.clone() for x in xs], [], []
    block(bb, torch, ins[0], ws)
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(block(bb, torch, ins[i], ws))
        graphs.append(g)
    for turn in range(4):
        for i in range(2):
            x = torch.randn(m, 256, generator=generator(torch, 10 * turn + i), device="cuda")
            ins[i].copy_(x)
            graphs[i].replay()
            want = block(bb, torch, x, ws)
            torch.cuda.synchronize()
            for a, b in zip(outs[i], want):
                assert torch.equal(a, b)


def test_block_on_streams(torch):
    """Calls on two streams at once, the streams given by name, give the sequential results."""
    ws = block_weights(torch, 256, 640, 777, 3)
    xs = [torch.randn(m, 256, generator=generator(torch, m), device="cuda") for m in (3, 90, 200)]
    want = [block(bb, torch, x, ws) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for turn in range(6):
        st = streams[turn % 2]
        x = xs[turn % 3]
        c, s = bb.quantize_fp8(x, stream=st)
        h, hs = bb.fp8_gemm_gated_quantize(c, s, ws[0], ws[1], stream=st)
        y = bb.fp8_gemm(h, hs, ws[2], dtype=torch.bfloat16, stream=st)
        with torch.cuda.stream(st):
            z = x + y
        c, s = bb.quantize_fp8(z, stream=st)
        logits = bb.fp8_gemm(c, s, ws[3], stream=st)
        got.append((z, logits) + bb.token_logprobs(logits, topk=4, stream=st)[1:])
    torch.cuda.synchronize()
    for turn, parts in enumerate(got):
        for a, b in zip(parts, want[turn % 3]):
            assert torch.equal(a, b)


PARTS = [(300, 256, 8192), (300, 520, 120 * 128 + 32)]  # over parts of K, through a workspace


def test_parts_of_k_from_graphs_and_threads(torch):
    """Calls that need a workspace: two graphs' replays, then two threads on streams of their own,
    with eager calls between, give the same bits."""
    for m, n, k in PARTS:
        assert "parts of K" in bb.fp8_gemm_kernel_name(m, n, k, torch.bfloat16)
        g = generator(torch, m)
        c, s = real_codes(torch, g, m, k, 1, False)
        w = [bb.Fp8Weights(*real_codes(torch, g, n, k, 128, False)) for _ in range(2)]
        want = [bb.fp8_gemm(c, s, v, dtype=torch.bfloat16) for v in w]
        torch.cuda.synchronize()
        graphs, outs = [], []
        for v in w:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                outs.append(bb.fp8_gemm(c, s, v, dtype=torch.bfloat16))
            graphs.append(gr)
        for _ in range(4):
            for i in range(2):
                outs[i].fill_(0)
                graphs[i].replay()
                again = bb.fp8_gemm(c, s, w[1 - i], dtype=torch.bfloat16)
                torch.cuda.synchronize()
                assert torch.equal(outs[i], want[i]) and torch.equal(again, want[1 - i])
        got = [[], []]

        def work(i):
            st = torch.cuda.Stream()
            for _ in range(20):
                got[i].append(bb.fp8_gemm(c, s, w[i], dtype=torch.bfloat16, stream=st))
            st.synchronize()
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        for i in range(2):
            assert len(got[i]) == 20 and all(torch.equal(y, want[i]) for y in got[i])


def test_one_matrix_for_both_projections(torch):
    for m, f, k in ((3, 160, 256), (70, 320, 416), (300, 2048, 288)):
        g = generator(torch, f)
        c, s = real_codes(torch, g, m, k, 1, False)
        w = bb.Fp8Weights(*real_codes(torch, g, f, k, 128, False))
        other = bb.Fp8Weights(w.codes.clone(), w.scales.clone())
        for dt in (torch.float32, torch.bfloat16):
            assert torch.equal(bb.fp8_gemm_gated(c, s, w, w, dtype=dt),
                               bb.fp8_gemm_gated(c, s, w, other, dtype=dt))
        for a, b in zip(bb.fp8_gemm_gated_quantize(c, s, w, w),
                        bb.fp8_gemm_gated_quantize(c, s, w, other)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("m,n,k", [(3, 150, 544), (40, 260, 672), (70, 1300, 800), (270, 300, 1056),
                                   (2050, 4100, 416), (300, 256, 8192)])
def test_nan_scale_stays_in_its_row_and_columns(torch, m, n, k):
    """A NaN among the scales reaches its row, or its 128 columns: scales of the blocks and rows
    beside a block are read along with its own."""
    for dt in (torch.float32, torch.bfloat16):
        g = generator(torch, k)
        c, s = real_codes(torch, g, m, k, 1, False)
        w = bb.Fp8Weights(*real_codes(torch, g, n, k, 128, False))
        s[1, 0] = math.nan
        s[m - 2, blocks(k) - 1] = math.nan
        w.scales[0, blocks(k) // 2] = math.nan
        y = torch.isnan(bb.fp8_gemm(c, s, w, dtype=dt))
        want = torch.zeros_like(y)
        want[1], want[m - 2], want[:, :128] = True, True, True
        assert torch.equal(y, want)


def test_inputs_that_require_gradients(torch):
    """Tensors that require gradients are read as values (the route is for inference)."""
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    codes, scales = bb.quantize_fp8(x)
    assert not scales.requires_grad


# ------------------------------------------------------------------ every plan, more blocks of K than 60

# gated: a wave loads the scales of both matrices anew every 60 blocks of K
GATED_LONG = [(18, 32, 61 * 128), (33, 64, 120 * 128 + 32), (39, 33, 61 * 128), (67, 4864, 61 * 128),
              (65, 4256, 120 * 128 + 32), (210, 4160, 61 * 128), (400, 4288, 61 * 128),
              (514, 3776, 120 * 128 + 32), (712, 2784, 61 * 128), (952, 4128, 61 * 128),
              (1171, 3309, 61 * 128), (1428, 3045, 120 * 128 + 32), (1557, 4832, 61 * 128),
              (1574, 4887, 61 * 128), (1844, 4640, 61 * 128), (2029, 4571, 61 * 128)]
# two kernels side by side that the shapes above do not reach
SIDE_BY_SIDE = [(2078, 8226, 2080), (3105, 5277, 32), (2178, 7196, 32), (5400, 1630, 288)]
GATED_SIDE_BY_SIDE = [(1611, 5326, 2080), (1812, 4447, 32), (2689, 3043, 32)]

# few rows of so many columns that they are made in tiles
FEW_OF_MANY = [(1, 17408, 160), (3, 17409, 96), (16, 20003, 1024), (9, 65540, 160), (16, 65539, 4128),
               (5, 131072, 544)]


@pytest.mark.parametrize("m,f,k", GATED_LONG + GATED_SIDE_BY_SIDE)
def test_gated_exact_relu_long_k(torch, m, f, k):
    """Codes of 1, 0 and -1 under scales of 1/4 to 4: both projections are whole multiples of 2^-4
    below 2^18, so their product rounds once."""
    g = generator(torch, m + f + k)
    c, s = small_codes(torch, g, m, k, 1), power_scales(torch, g, m, blocks(k))
    gate, up = (bb.Fp8Weights(small_codes(torch, g, f, k, 1),
                              power_scales(torch, g, blocks(f), blocks(k))) for _ in range(2))
    a = wide_values(torch, c, s, 1)
    wg, wu = (wide_values(torch, w.codes, w.scales, 128) for w in (gate, up))
    h = (torch.relu(mm64(torch, a, wg)) * mm64(torch, a, wu)).float()
    for dt in (torch.float32, torch.bfloat16):
        got = bb.fp8_gemm_gated(c, s, gate, up, activation="relu", dtype=dt)
        assert torch.equal(got, h.to(dt)), torch.nonzero(got != h.to(dt))[:4]
    if f % 32 == 0:
        codes, scales = bb.fp8_gemm_gated_quantize(c, s, gate, up, activation="relu")
        q, d = plain_codes(torch, h.cpu(), 1)
        assert torch.equal(scales.cpu(), d)
        assert torch.equal(codes.cpu().view(torch.uint8) & 0x7f, q & 0x7f)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n,k", SIDE_BY_SIDE + FEW_OF_MANY)
def test_product_exact_side_by_side(torch, m, n, k, dtype):
    dt = getattr(torch, dtype)
    g = generator(torch, m + n + k)
    c, s = small_codes(torch, g, m, k), power_scales(torch, g, m, blocks(k))
    w = bb.Fp8Weights(small_codes(torch, g, n, k), power_scales(torch, g, blocks(n), blocks(k)))
    got = bb.fp8_gemm(c, s, w, dtype=dt)
    ref = mm64(torch, wide_values(torch, c, s, 1), wide_values(torch, w.codes, w.scales, 128)).to(dt)
    assert torch.equal(got, ref), torch.nonzero(got != ref)[:4]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("m,f,k", [s for s in GATED if s[0] > 16] + [(0, 64, 64), (1, 64, 96)])
def test_exact_codes_are_those_of_the_fp32_values(torch, m, f, k, act):
    """exact=True, any number of rows: bit for bit the codes of the fp32 values, which lie within the
    fp32 products' bound of h (as in test_gated_quantize, without the 8-bit instruction's part)."""
    c, s, gate, up = gated_case(torch, max(m, 1), f, k, m + f + k)
    c, s = c[:m], s[:m]
    codes, scales = bb.fp8_gemm_gated_quantize(c, s, gate, up, activation=act, exact=True)
    want = bb.quantize_fp8(bb.fp8_gemm_gated(c, s, gate, up, activation=act))
    given = (torch.empty_like(codes), torch.empty_like(scales))
    again = bb.fp8_gemm_gated_quantize(c, s, gate, up, act, *given, exact=True)
    assert again[0] is given[0] and again[1] is given[1]
    for a, b, d in zip((codes, scales), want, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(a.view(torch.uint8), d.view(torch.uint8))
    if m == 0:
        return
    h, lim = gated_reference(torch, c, s, gate, up, act, True)
    d = scales.double().repeat_interleave(128, 1)[:, :f]
    size = h.abs() + lim
    step = torch.maximum(size * 2.0 ** -4, 2.0 ** -10 * d)
    assert ((codes.double() * d - h).abs() <= step + lim + 4 * U * size).all()


def test_exact_codes_from_graphs(torch):
    g = generator(torch, 8)
    m, f, k = 70, 320, 544
    c, s = real_codes(torch, g, m, k, 1, True)
    ws = [bb.Fp8Weights(*real_codes(torch, g, f, k, 128, False)) for _ in range(3)]
    calls = [lambda i=i: bb.fp8_gemm_gated_quantize(c, s, ws[i], ws[i + 1], exact=True) for i in range(2)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in calls:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call())
        graphs.append(gr)
    for _ in range(4):
        for i in range(2):
            for t in outs[i]:
                t.view(torch.uint8).fill_(0)
            graphs[i].replay()
            other = calls[1 - i]()
            torch.cuda.synchronize()
            for a, b in zip(outs[i] + other, want[i] + want[1 - i]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))

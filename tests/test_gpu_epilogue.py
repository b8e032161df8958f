"""The dense product with bias, activation and residual in its epilogue.

Bars: with an empty epilogue every element equals w4a4_gemm's (or its bf16
rounding) bit for bit, on every kernel a dense product runs; otherwise each
element lies within the fp32 bound of the product, carried through the
activation's slope, plus the roundings of the epilogue's own steps, of the
64-bit formula on the oracle's product.
"""
import math

import numpy as np
import pytest

import oracle
from bit_prefill_gemm_amd import binding as bb
from bit_prefill_gemm_amd import synth

from gpu_util import act_to_device, assert_within_bound, fp32_bound, oracle_codes, rects, torch_mod

pytestmark = pytest.mark.gpu

# m, k, n, bits, kernel: every kernel an epilogue runs, odd rows, K that ends inside a group and a
# stage; chunks of 16 rows: one row more than a chunk, K with and without staged rows, K of one
# block, the most tiles on both sides of K = 2048, and one tile more
CASES = [
    (1, 1024, 4128, 4, "weight-stream"), (1, 1056, 4128, 8, "weight-stream"),
    (16, 416, 4160, 4, "weight-stream"), (9, 8192, 4128, 8, "weight-stream"),
    # one row and half tiles (at most 128 tiles of 32 columns), whole ones
    (1, 1024, 96, 4, "weight-stream chunks"), (1, 1056, 64, 8, "weight-stream chunks"),
    (16, 2080, 160, 4, "weight-stream chunks"), (9, 8192, 64, 8, "weight-stream chunks"),
    (16, 96, 4096, 4, "weight-stream chunks"), (64, 1024, 1024, 8, "weight-stream chunks"),
    (65, 1024, 1024, 4, "weight-stream chunks"),
    (13, 32800, 32, 4, "tiled 16x32"), (9, 32800, 64, 8, "tiled 16x32"),
    (1025, 96, 2176, 4, "strip 32x128"), (1030, 160, 2176, 8, "strip 32x128"),
    # strips over widths that leave one, two and three of the last strip's tiles
    (640, 416, 2080, 4, "strip 32x128"), (601, 1056, 2112, 8, "strip 32x128"), (650, 96, 2144, 4, "strip 32x128"),
    (512, 1056, 5120, 4, "wide 64x160"), (512, 544, 5120, 4, "strip 32x128"),
    (449, 4128, 5120, 8, "tiled 64x160"), (1025, 96, 576, 4, "tiled 64x32"),
    (1041, 2080, 1056, 4, "tiled 64x32"), (520, 96, 1056, 8, "tiled 64x32"),
    (17, 1024, 128, 8, "weight-stream chunks"), (31, 96, 64, 4, "weight-stream chunks"),
    (33, 416, 128, 4, "weight-stream chunks"), (100, 1056, 256, 8, "weight-stream chunks"),
    (77, 2080, 1056, 8, "weight-stream chunks"), (300, 32, 96, 4, "weight-stream chunks"),
    (40, 6560, 64, 4, "weight-stream chunks"), (50, 4000, 32, 8, "weight-stream chunks"),
    (1024, 64, 512, 4, "weight-stream chunks"), (1025, 64, 512, 4, "tiled 64x32"),
    (512, 2048, 2048, 4, "weight-stream chunks"), (513, 2048, 2048, 4, "tiled 64x32"),
    (20, 32768, 32, 4, "weight-stream chunks"), (20, 32800, 32, 4, "tiled 64x32"),
]


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    return t


def host(t):
    torch = torch_mod()
    t = t.cpu().contiguous()
    return synth.bf16_to_f32(t.view(torch.int16).numpy().view(np.uint16)) if t.dtype == torch.bfloat16 else t.numpy()


_made = {}


def problem(m, k, n, bits, rotation=32):
    """Codes, image, and the oracle's product (fp64) with its absolute sum, made once a shape."""
    torch = torch_mod()
    key = (m, k, n, bits, rotation)
    if key not in _made:
        rng = np.random.default_rng(m + k + n + bits)
        x = rng.standard_normal((m, k)).astype(np.float32)
        q, d, _ = oracle.quantize(x, bits)
        # unit-sized results, so that activations are met where they bend
        blocks = synth.draw_q4_0(rng, (n,), k, 0.02 / math.sqrt(k), 0.6 / math.sqrt(k))
        pack = bb.pack_weights_unrotated if rotation == 0 else bb.rotate_pack_weights
        kind = bb.SRC_Q4_0 if rotation == 0 else bb.SRC_Q4_0_ROTATED
        W = pack(blocks, kind, n, k).to("cuda")
        w, dw = oracle.q4_0_decode(blocks, k)
        codes = torch.from_numpy(oracle_codes(q, bits)).cuda()
        scales = torch.from_numpy(d).cuda()
        ref = oracle.gemm_rect(q, d, w, dw, 0, m, 0, n)
        mag = oracle.gemm_abs_rect(q, d, w, dw, 0, m, 0, n)
        _made[key] = codes, scales, W, ref, mag
    return _made[key]


def erf64(x):
    return np.vectorize(math.erf, otypes=[np.float64])(x)


def act64(t, act):
    if act == "relu":
        return np.maximum(t, 0.0)
    if act == "silu":
        return t / (1.0 + np.exp(-t))
    if act == "gelu":
        return 0.5 * t * (1.0 + erf64(t / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * t * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (t + 0.044715 * t ** 3)))
    return t


def limit(mag, k, t, y, out, act, bias, residual):
    """The element-wise bound.  t carries the product's fp32 bound and the bias's rounding; an
    activation's slope is at most 1.13; its own steps (an exponential or erf within 2 ulp, a sum,
    a quotient, a product, and for the tanh form the argument's four roundings, which enter
    through |z| sigmoid'(z) <= 0.23) stay below 12 2^-24 |t|; the residual's addition and the
    output's rounding are half a step each."""
    u = 2.0 ** -24
    lim = fp32_bound(mag, k)
    if bias:
        lim = lim + u * np.abs(t)
    if act not in ("none", "relu"):
        lim = 1.13 * lim + 12 * u * np.abs(t)
    if residual:
        lim = lim + u * np.abs(y)
    lim = lim * (1 + 2.0 ** -16)
    return lim if out == "fp32" else lim + 2.0 ** -8 * (np.abs(y) + lim)


def check(torch, case, act="none", bias=None, residual=None, out="fp32", pads=(0, 0), in_place=False):
    m, k, n, bits = case[:4]
    codes, scales, W, ref, mag = problem(m, k, n, bits)
    assert bb.w4a4_gemm_epilogue_kernel_name(bits, m, W) == case[4]
    print("epilogue", case, act, bias, residual, out, flush=True)
    rng = np.random.default_rng(n + m)
    types = {"fp32": torch.float32, "bf16": torch.bfloat16}
    b = r = None
    if bias:
        b = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda().to(types[bias])
    if residual:
        r = torch.full((m, n + pads[0]), 7.0, dtype=types[residual], device="cuda")
        r[:, :n] = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).cuda()
        r = r[:, :n]
    t = ref + (0.0 if b is None else host(b).astype(np.float64))
    y64 = act64(t, act) + (0.0 if r is None else host(r).astype(np.float64))
    wide = r if in_place else torch.full((m, n + pads[1]), 5.0, dtype=types[out], device="cuda")
    y = bb.w4a4_gemm_epilogue(codes, scales, bits, W, bias=b, activation=act, residual=r, y=wide[:, :n])
    torch.cuda.synchronize()
    if not in_place:
        assert (wide[:, n:] == 5.0).all()
        if r is not None and pads[0]:
            assert (r.as_strided((m, n + pads[0]), r.stride())[:, n:] == 7.0).all()
    err = np.abs(host(y).astype(np.float64) - y64)
    lim = limit(mag, k, t, y64, out, act, b is not None, r is not None)
    bad = np.argwhere(~(err <= lim))
    assert bad.size == 0, "%d elements, first %s: %g > %g" % (
        len(bad), bad[0].tolist(), err[tuple(bad[0])], lim[tuple(bad[0])])


@pytest.mark.parametrize("case", CASES, ids=["%dx%dx%d-%d" % c[:4] for c in CASES])
def test_empty_epilogue_is_the_product(torch, case):
    m, k, n, bits, kernel = case
    codes, scales, W, _, _ = problem(m, k, n, bits)
    assert bb.w4a4_gemm_epilogue_kernel_name(bits, m, W) == kernel
    y = bb.w4a4_gemm_epilogue(codes, scales, bits, W)
    if bb.w4a4_gemm_kernel_name(bits, m, W) == kernel:
        assert torch.equal(y, bb.w4a4_gemm(codes, scales, bits, W))
    # bf16 output is the fp32 result rounded, and every run gives the same bits
    assert torch.equal(bb.w4a4_gemm_epilogue(codes, scales, bits, W, dtype=torch.bfloat16), y.bfloat16())
    assert torch.equal(bb.w4a4_gemm_epilogue(codes, scales, bits, W), y)


@pytest.mark.parametrize("case", CASES, ids=["%dx%dx%d-%d" % c[:4] for c in CASES])
def test_every_step_on_every_kernel(torch, case):
    check(torch, case, "silu", "fp32", "bf16", "bf16")
    check(torch, case, "gelu", "bf16", "fp32", "fp32", pads=(3, 16))
    check(torch, case, "gelu_tanh", "fp32", None, "fp32")
    check(torch, case, "relu", None, "fp32", "bf16", pads=(5, 8))
    check(torch, case, "none", "bf16", "bf16", "fp32", pads=(1, 4))
    # the residual stream updated where it is
    check(torch, case, "none", None, "bf16", "bf16", in_place=True)
    check(torch, case, "silu", "fp32", "fp32", "fp32", in_place=True)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("kind", [None, "fp32", "bf16"])
def test_activations_and_types(torch, act, kind):
    for case in ((17, 1024, 128, 8, "weight-stream chunks"), (650, 96, 2144, 4, "strip 32x128")):
        check(torch, case, act, kind, None, "fp32")
        check(torch, case, act, None, kind, "bf16")


def test_activations_far_out(torch):
    """Arguments far from zero: the activations reach 0 and x, never NaN, and stay as exact as near zero."""
    case = (33, 416, 128, 4, "weight-stream chunks")
    m, k, n, bits = case[:4]
    codes, scales, W, ref, mag = problem(m, k, n, bits)
    bias = torch.linspace(-200.0, 200.0, n, device="cuda")
    bias[0], bias[1], bias[2], bias[3] = -3e38, 3e38, -90.0, -104.0
    t = ref + host(bias).astype(np.float64)
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        y = host(bb.w4a4_gemm_epilogue(codes, scales, bits, W, bias=bias, activation=act)).astype(np.float64)
        with np.errstate(over="ignore", invalid="ignore"):
            y64 = act64(t, act)
        y64 = np.where(np.isnan(y64), 0.0, y64)
        big = np.abs(t) > 1e30
        lim = limit(mag, k, t, y64, "fp32", act, True, False)
        assert (np.abs(y - y64)[~big] <= lim[~big]).all(), act
        assert (np.abs(y - y64)[big] <= 1e-6 * np.abs(t[big])).all(), act


def random_weights(torch, n, k, seed):
    """An image of random codes and scales, made on the GPU (its layout is the packer's)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    groups = (k // 32 + 3) // 4
    img = torch.randint(0, 256, (n // 32 * groups, 2304), dtype=torch.uint8, device="cuda", generator=g)
    scale = (0.002 + 0.018 * torch.rand(n // 32 * groups, 128, device="cuda", generator=g)).half()
    img[:, 2048:] = scale.view(torch.uint8)
    d = bb.WeightsDesc(0x57475042, 1, 32, 3, n, k, 1, img.numel(), 2048)
    return bb.Weights(d, img.view(-1))


@pytest.mark.parametrize("m,k,n,bits,kernel", [(9, 32896, 16448, 4, "tiled 16x64"), (3, 32896, 16448, 8, "tiled 16x64"),
                                               (25, 512, 16640, 4, "weight-stream"), (32, 1024, 16640, 8, "weight-stream"),
                                               (500, 1024, 5120, 4, "wide 64x160")])
def test_steps_on_the_products_own_result(torch, m, k, n, bits, kernel):
    """Where both entry points run the same kernel, bias, relu and residual are single fp32
    operations on w4a4_gemm's result: equal bit for bit."""
    W = random_weights(torch, n, k, m)
    assert bb.w4a4_gemm_epilogue_kernel_name(bits, m, W) == kernel == bb.w4a4_gemm_kernel_name(bits, m, W)
    print("own result", m, k, n, bits, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + 1)
    x = torch.randn(m, k, device="cuda", generator=g)
    codes, scales = bb.quantize_act_h32(x, bits)
    t = bb.w4a4_gemm(codes, scales, bits, W)
    bias = torch.randn(n, device="cuda", generator=g)
    res = torch.randn(m, n, device="cuda", generator=g).bfloat16()
    y = bb.w4a4_gemm_epilogue(codes, scales, bits, W, bias=bias, activation="relu", residual=res)
    assert torch.equal(y, torch.relu(t + bias) + res.float())
    y = bb.w4a4_gemm_epilogue(codes, scales, bits, W, residual=res, dtype=torch.bfloat16)
    assert torch.equal(y, (t + res.float()).bfloat16())


def test_unrotated_and_stamps(torch):
    m, k, n, bits = 5, 256, 64, 4
    codes, scales, W, ref, mag = problem(m, k, n, bits, rotation=0)
    y = host(bb.w4a4_gemm_epilogue(codes, scales, bits, W, rotation=0))
    assert (np.abs(y - ref) <= fp32_bound(mag, k) * (1 + 2.0 ** -20)).all()
    assert np.array_equal(y, host(bb.w4a4_gemm_unrotated(codes, scales, bits, W)))
    for rotation in (32, 64, 128):
        with pytest.raises(bb.BpgError) as e:
            bb.w4a4_gemm_epilogue(codes, scales, bits, W, rotation=rotation)
        assert e.value.status == 5


def test_rows_behind_stay(torch):
    """Rows of y and of the residual behind the last token are not touched."""
    for case in CASES[2:]:
        m, k, n, bits = case[:4]
        codes, scales, W, _, _ = problem(m, k, n, bits)
        y = torch.full((m + 40, n), 9.0, device="cuda")
        bb.w4a4_gemm_epilogue(codes, scales, bits, W, residual=y[:m], y=y[:m], activation="silu")
        assert (y[m:] == 9.0).all()


def test_no_rows(torch):
    _, _, W, _, _ = problem(5, 256, 64, 4)
    y = bb.w4a4_gemm_epilogue(torch.empty(0, 128, dtype=torch.uint8, device="cuda"),
                              torch.empty(0, 8, device="cuda"), 4, W,
                              residual=torch.empty(0, 64, device="cuda"), bias=torch.zeros(64, device="cuda"))
    assert y.shape == (0, 64)


# every kernel that an epilogue runs, the weight-stream one with one and two row tiles
TAILS = [(16, 512, 16416, 4, "weight-stream"), (25, 512, 16640, 4, "weight-stream"),
         (33, 416, 128, 4, "weight-stream chunks"), (650, 96, 2144, 4, "strip 32x128"),
         (601, 1056, 2112, 8, "strip 32x128"), (512, 1056, 5120, 4, "wide 64x160"),
         (449, 4128, 5120, 8, "tiled 64x160"), (1025, 96, 576, 4, "tiled 64x32")]


def own_result(torch, case, act):
    """(t, y), where the product is exactly 0 (all codes are), so that t is the bias itself."""
    m, k, n, bits, kernel = case
    W = random_weights(torch, n, k, 1)
    assert bb.w4a4_gemm_epilogue_kernel_name(bits, m, W) == kernel
    print("tails", case, act, flush=True)
    t = np.random.default_rng(n).permutation(np.linspace(-130.0, 20.0, n)).astype(np.float32)
    t[:8] = -5.5, -12.5, -90.0, -104.0, 1e-30, -1e-30, -1e30, 0.0
    codes = torch.zeros(m, k * bits // 8, dtype=torch.uint8, device="cuda")
    scales = torch.ones(m, k // 32, device="cuda")
    y = bb.w4a4_gemm_epilogue(codes, scales, bits, W, bias=torch.from_numpy(t).cuda(), activation=act)
    assert (y == y[0]).all()
    return t.astype(np.float64), host(y[0]).astype(np.float64)


def off(y, y64, relative, absolute):
    err, lim = np.abs(y - y64), (relative * np.abs(y64) + absolute) * (1 + 2.0 ** -10)
    bad = np.flatnonzero(~(err <= lim))
    return [(y[i], y64[i], err[i] / lim[i]) for i in bad[:5]]


@pytest.mark.parametrize("case", TAILS, ids=["%dx%dx%d-%d" % c[:4] for c in TAILS])
def test_gelu_tail(torch, case):
    """GELU relative to its result, down to where erfc leaves fp32's normal numbers (below them
    erfc may be 0: times |t| / 2 < 8 that is 2^-123).  y = t / 2 erfc(x), x = -t / sqrt 2 with the
    constant's rounding and the product's (1.3 2^-24), which enter times
    |d ln erfc / d ln x| <= x (x + sqrt(x^2 + 2)) <= t^2 + 1; erfc within the 16 ulp that OpenCL
    asks of it (32 2^-24), and a product's rounding."""
    t, y = own_result(torch, case, "gelu")
    y64 = 0.5 * t * np.vectorize(math.erfc, otypes=[np.float64])(-t / math.sqrt(2.0))
    assert off(y, y64, 2.0 ** -24 * (33 + 1.3 * (np.minimum(t * t, 200.0) + 1)), 2.0 ** -123) == []


@pytest.mark.parametrize("case", TAILS, ids=["%dx%dx%d-%d" % c[:4] for c in TAILS])
def test_silu_tail(torch, case):
    """SiLU relative to its result, down to fp32's subnormal numbers: the sigmoid within 8 2^-24
    and a product's rounding; a subnormal result is rounded to a multiple of 2^-149 at most twice."""
    t, y = own_result(torch, case, "silu")
    with np.errstate(over="ignore"):
        y64 = t / (1.0 + np.exp(-t))
    assert off(y, y64, 9 * 2.0 ** -24, 2.0 ** -149) == []


@pytest.mark.parametrize("case", TAILS, ids=["%dx%dx%d-%d" % c[:4] for c in TAILS])
def test_gelu_tanh_tail(torch, case):
    """As SiLU at z = 2 sqrt(2 / pi) (t + 0.044715 t^3), whose roundings are within 7 2^-24 (the
    cubic's constant and three products, a sum, the factor's constant and its product) and enter
    times |d ln sigmoid / d ln z| <= |z|; beyond |z| = 150 the result is 0 or t."""
    t, y = own_result(torch, case, "gelu_tanh")
    z = 2.0 * math.sqrt(2.0 / math.pi) * (t + 0.044715 * t ** 3)
    with np.errstate(over="ignore"):
        y64 = t / (1.0 + np.exp(-z))
    assert off(y, y64, 2.0 ** -24 * (9 + 7 * np.minimum(np.abs(z), 150.0)), 2.0 ** -149) == []


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("case", TAILS, ids=["%dx%dx%d-%d" % c[:4] for c in TAILS])
def test_far_values_leave_the_others_their_bits(torch, case, act):
    """Alone in its columns' wave or beside values far out, a value's result is the same."""
    m, k, n, bits = case[:4]
    W = random_weights(torch, n, k, 2)
    codes = torch.zeros(m, k * bits // 8, dtype=torch.uint8, device="cuda")
    scales = torch.ones(m, k // 32, device="cuda")
    near = torch.from_numpy(np.random.default_rng(m).uniform(-60.0 if act == "silu" else -8.0, 20.0, n).astype(np.float32)).cuda()
    far = near.clone()
    at = torch.arange(n, device="cuda") % 3 == 0
    far[at] = torch.linspace(-130.0, -9.0, int(at.sum()), device="cuda")
    print("neighbours", case, act, flush=True)
    a = bb.w4a4_gemm_epilogue(codes, scales, bits, W, bias=near, activation=act)
    b = bb.w4a4_gemm_epilogue(codes, scales, bits, W, bias=far, activation=act)
    assert torch.equal(a[:, ~at], b[:, ~at]) and not torch.equal(a[:, at], b[:, at])


# two row tiles of the weight-stream kernel: 17 to 32 rows past the chunks' bound
TWO_ROW_TILES = [(25, 416, 16416, 4, "weight-stream"), (32, 96, 16448, 8, "weight-stream"),
                 (17, 1056, 16512, 8, "weight-stream")]


@pytest.mark.parametrize("case", TWO_ROW_TILES, ids=["%dx%dx%d-%d" % c[:4] for c in TWO_ROW_TILES])
def test_every_step_on_two_row_tiles(torch, case):
    test_empty_epilogue_is_the_product(torch, case)
    test_every_step_on_every_kernel(torch, case)


@pytest.mark.parametrize("m,k,n,bits,kernel", [(1, 2048, 5120, 4, "weight-stream"), (25, 512, 16640, 8, "weight-stream"),
                                               (40, 384, 96, 4, "weight-stream chunks"), (700, 128, 2144, 8, "strip 32x128"),
                                               (500, 1024, 5120, 4, "wide 64x160"), (449, 4096, 5120, 8, "tiled 64x160"),
                                               (1025, 128, 576, 4, "tiled 64x32")])
@pytest.mark.parametrize("rotation", [64, 128])
def test_longer_rotations(torch, rotation, m, k, n, bits, kernel):
    """Codes and weights of the longer spans, through their own quantizer and packer: the product
    within its fp32 bound of the 64-bit one of the same codes, and, with bias, activation and
    residual, the bits that the same image and codes give where the stamp says 32."""
    rng = np.random.default_rng(m + rotation)
    blocks = synth.draw_q4_0(rng, (n,), k, 0.02 / math.sqrt(k), 0.6 / math.sqrt(k))
    W = bb.rotate_pack_weights_rot(blocks, bb.SRC_Q4_0_ROTATED, n, k, rotation).to("cuda")
    assert W.desc.rotation == rotation and bb.w4a4_gemm_epilogue_kernel_name(bits, m, W) == kernel
    print("rotation", rotation, m, k, n, bits, flush=True)
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).cuda()
    codes, scales = bb.quantize_act_rot(x, rotation, bits)
    y = bb.w4a4_gemm_epilogue(codes, scales, bits, W, rotation=rotation)
    if bb.w4a4_gemm_kernel_name(bits, m, W) == kernel:
        assert torch.equal(y, bb.w4a4_gemm_rot(codes, scales, bits, rotation, W))
    # the codes themselves: their values at scales of 1, not rotated back
    q = host(bb.dequantize_act(codes, torch.ones_like(scales), bits, 0)).astype(np.int8)
    w, dw = oracle.q4_0_decode(blocks, k)
    for m0, m1, n0, n1 in rects(m, n, 96, 3, rotation):
        ref = oracle.gemm_rect(q, host(scales), w, dw, m0, m1, n0, n1)
        mag = oracle.gemm_abs_rect(q, host(scales), w, dw, m0, m1, n0, n1)
        assert_within_bound(host(y)[m0:m1, n0:n1], ref, mag, k, "rotation %d" % rotation)
    bias = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    res = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).cuda().bfloat16()
    steps = dict(bias=bias, activation="gelu_tanh", residual=res, dtype=torch.bfloat16)
    got = bb.w4a4_gemm_epilogue(codes, scales, bits, W, rotation=rotation, **steps)
    plain = bb.WeightsDesc.from_buffer_copy(W.desc)
    plain.rotation = 32
    assert torch.equal(got, bb.w4a4_gemm_epilogue(codes, scales, bits, bb.Weights(plain, W.image), **steps))
    with pytest.raises(bb.BpgError) as e:
        bb.w4a4_gemm_epilogue(codes, scales, bits, W, rotation=32)
    assert e.value.status == 5

"""RMSNorm + residual + rotation + quantization, and the decoding of codes.

Bars: the new stream h, the codes and the scales are equal bit for bit to a
plain evaluation of the definition (numpy fp32 steps and a 64-bit sum, then the
oracle's quantizer); every decoded value lies within half a quantization step
of the 64-bit formula plus the fp32 roundings on the way; decoded values are
equal bit for bit to the oracle's rotation of code * scale.
"""
import numpy as np
import pytest

import oracle
from bit_prefill_gemm_amd import binding as bb
from bit_prefill_gemm_amd import synth

from gpu_util import act_to_device, oracle_codes, torch_mod

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    return t


def f32(a):
    return a if a.dtype == np.float32 else synth.bf16_to_f32(a)


def to_type(v, like):
    """fp32 values rounded to the type of `like` (fp32, or bf16 bits)."""
    return v if like.dtype == np.float32 else synth.bf16_bits(v)


def host(t):
    torch = torch_mod()
    t = t.cpu().contiguous()
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()


def padded(torch, a, pad):
    """A device tensor of `a` whose rows are `pad` elements apart from each other."""
    t = act_to_device(a)
    if not pad:
        return t
    wide = torch.full((a.shape[0], a.shape[1] + pad), 3.0, dtype=t.dtype, device="cuda")
    wide[:, :a.shape[1]] = t
    return wide[:, :a.shape[1]]


def expected(x, r, w, eps):
    """(h in the stream's type, v fp32): the definition, step by step."""
    h = x if r is None else to_type(f32(x) + f32(r), r)
    f = f32(h)
    ss = np.sum(f.astype(np.float64) ** 2, axis=1)
    s = (1.0 / np.sqrt(ss / f.shape[1] + np.float64(np.float32(eps)))).astype(np.float32)
    v = f * s[:, None]
    return h, (v if w is None else v * f32(w)[None, :])


def quantized(v, bits, rot):
    if rot > 32:
        return oracle.quantize_rot(v, rot, bits)[:2]
    return oracle.quantize(v, bits, rotate=rot != 0)[:2]


def check_formula(h, w, eps, bits, rot, q, d):
    """|q d - v| <= d / 2 + roundings, v the formula in 64 bits in the rotated basis.  Before the
    rotation a value carries the roundings of s, h s and (h s) g (3 halves of 2^-23); each of the
    log2(rot) stages and the factor (rounded constant and product) adds one rounding of a number
    of at most sum |v| over the span, /sqrt(rot) after the factor; d carries one rounding, q d one,
    and the quotient v / d one of at most 127.5 2^-24 steps."""
    f = f32(h).astype(np.float64)
    v = f / np.sqrt(np.mean(f * f, axis=1, keepdims=True) + np.float64(np.float32(eps)))
    if w is not None:
        v = v * f32(w).astype(np.float64)
    m, k = v.shape
    u = 2.0 ** -24
    if rot:
        mag = np.repeat(np.abs(v).reshape(m, -1, rot).sum(2) / np.sqrt(rot), rot, axis=1)
        stages = int(np.log2(rot))
        v = oracle.rotate_n_f64(v, rot) if rot != 32 else oracle.rotate_f64(v)
        slack = (3 + stages + 2) * u * mag
    else:
        slack = 3 * u * np.abs(v)
    dd = np.repeat(d.astype(np.float64), 32, axis=1)
    err = np.abs(q * dd - v)
    lim = dd * (0.5 + 130 * u) + 1.01 * slack + 2 * u * np.abs(v)
    bad = np.argwhere(err > lim)
    assert bad.size == 0, (bad[:3].tolist(), err.max())


def check(torch, x, r, w, bits, rot, eps=EPS, pads=(0, 0, 0), in_place=False):
    xd, rd = padded(torch, x, pads[0]), None if r is None else padded(torch, r, pads[1])
    wd = None if w is None else act_to_device(w[None, :])[0].contiguous()
    hd = None
    if r is not None and in_place:
        hd = rd
    elif r is not None and pads[2]:
        hd = padded(torch, np.zeros_like(r), pads[2])
    h, codes, scales = bb.rmsnorm_quantize_act(xd, residual=rd, weight=wd, eps=eps, act_bits=bits,
                                               rotation=rot, h=hd)
    torch.cuda.synchronize()
    ref_h, v = expected(x, r, w, eps)
    q, d = quantized(v, bits, rot)
    assert np.array_equal(host(h).view(np.uint8), ref_h.view(np.uint8)), "h differs"
    assert np.array_equal(host(scales).view(np.uint32), d.view(np.uint32)), "scales differ"
    bad = np.argwhere(host(codes) != oracle_codes(q, bits))
    assert bad.size == 0, "codes differ at %s (of %d)" % (bad[:5].tolist(), len(bad))
    for t, pad in ((xd, pads[0]), (rd, pads[1]), (hd, pads[2])):
        if t is not None and pad and t.shape[0] and not (in_place and t is rd):
            wide = t.as_strided((t.shape[0], t.shape[1] + pad), t.stride())
            assert (wide[:, t.shape[1]:] == 3.0).all(), "columns behind the rows were written"
    check_formula(ref_h, w, eps, bits, rot, q, d)
    return codes, scales, q, d


def draw(rng, m, k, dtype, outliers=True):
    x, _ = synth.draw_activations(rng, m, k, "normal", 0.01 if outliers else 0.0, 20.0)
    return x if dtype == "fp32" else synth.bf16_bits(x)


# one 32-block; one wave's end and one more block; every count of rounds per quad (1, 2, 4, 8)
# and its ends; the repository's widths; the largest row
SHAPES = [(1, 32), (3, 512), (5, 544), (7, 2080), (2, 5120), (3, 8192), (2, 8224), (2, 16384),
          (3, 16416), (1, 17408), (1, 32768), (2, 32800), (1, 65536), (301, 256), (1200, 96)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m,k", SHAPES)
def test_shapes(torch, m, k, bits):
    print("norm", m, k, bits, flush=True)
    rng = np.random.default_rng(m * 7 + k + bits)
    x, r = draw(rng, m, k, "bf16"), draw(rng, m, k, "bf16")
    w = synth.bf16_bits((1 + 0.1 * rng.standard_normal(k)).astype(np.float32))
    check(torch, x, r, w, bits, 32)


@pytest.mark.parametrize("rot", [0, 32, 64, 128])
@pytest.mark.parametrize("xt,rt,wt", [("fp32", "fp32", "fp32"), ("bf16", "fp32", "bf16"),
                                      ("fp32", "bf16", "fp32"), ("bf16", "bf16", None),
                                      ("fp32", None, "bf16"), ("bf16", None, "fp32")])
def test_types_and_spans(torch, xt, rt, wt, rot):
    for bits, (m, k) in ((4, (9, 640)), (8, (4, 1152)), (4, (2, 9216))):
        print("norm types", xt, rt, wt, rot, bits, flush=True)
        rng = np.random.default_rng(rot + bits + m)
        x = draw(rng, m, k, xt)
        r = None if rt is None else draw(rng, m, k, rt)
        w = None
        if wt is not None:
            w = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
            w = w if wt == "fp32" else synth.bf16_bits(w)
        check(torch, x, r, w, bits, rot)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides_and_in_place(torch, dtype):
    rng = np.random.default_rng(3)
    m, k = 17, 1056
    x, r = draw(rng, m, k, dtype), draw(rng, m, k, dtype)
    check(torch, x, r, None, 4, 32, pads=(4, 20, 36))
    check(torch, x, r, None, 8, 0, pads=(0, 12, 0), in_place=True)
    check(torch, x, r, None, 8, 32, in_place=True)
    check(torch, x, None, None, 4, 32, pads=(28, 0, 0))
    # one row of a wider buffer: its stride is free
    big = act_to_device(draw(rng, 1, 2 * k + 2, dtype))
    row = big[:, :k]
    h, codes, scales = bb.rmsnorm_quantize_act(row, residual=row, act_bits=4)
    ref_h, v = expected(host(row), host(row), None, 1e-6)
    q, d = quantized(v, 4, 32)
    assert np.array_equal(host(h), ref_h) and np.array_equal(host(codes), oracle_codes(q, 4))


def test_many_rows_walk_the_grid(torch):
    """More rows than workgroups (2^20): rows far apart are right, and none is left out."""
    m, k = (1 << 20) + 1000, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, k, device="cuda", generator=g)
    h, codes, scales = bb.rmsnorm_quantize_act(x, act_bits=8)
    assert h is x
    rows = np.r_[0:300, (1 << 20) - 300:m]
    sub = host(x[torch.from_numpy(rows).cuda()])
    _, v = expected(sub, None, None, 1e-6)
    q, d = quantized(v, 8, 32)
    assert np.array_equal(host(codes)[rows], oracle_codes(q, 8))
    assert np.array_equal(host(scales)[rows], d)
    assert int((scales > 0).sum()) == m


@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", None)])
def test_more_rows_than_fit_at_once(torch, xt, rt):
    """Workgroups that walk several rows, one to eight blocks per quad, the rows' loads ahead or not."""
    for m, k, bits in ((8200, 64, 4), (2000, 544, 4), (1700, 2048, 8), (1300, 8224, 4), (300, 17408, 4),
                       (270, 32768, 8), (260, 33792, 4)):
        print("norm many rows", xt, rt, m, k, bits, flush=True)
        g = torch.Generator(device="cuda").manual_seed(m + k)
        types = {"bf16": torch.bfloat16, "fp32": torch.float32}
        x = torch.randn(m, k, device="cuda", generator=g).to(types[xt])
        r = None if rt is None else torch.randn(m, k, device="cuda", generator=g).to(types[rt])
        w = torch.rand(k, device="cuda", generator=g)
        h, codes, scales = bb.rmsnorm_quantize_act(x, residual=r, weight=w, act_bits=bits)
        rows = np.unique(np.r_[0:3, m // 2, m - 40:m:7, m - 1, 255, 256, min(m - 1, 1024)])
        at = torch.from_numpy(rows).cuda()
        ref_h, v = expected(host(x[at]), None if r is None else host(r[at]), host(w), 1e-6)
        q, d = quantized(v, bits, 32)
        assert np.array_equal(host(h[at]), ref_h)
        assert np.array_equal(host(codes[at]), oracle_codes(q, bits)) and np.array_equal(host(scales[at]), d)


def test_zero_tiny_and_huge_rows(torch):
    k = 256
    rng = np.random.default_rng(5)
    x = rng.standard_normal((8, k)).astype(np.float32)
    x[0] = 0.0                       # scale 0, codes 0
    x[1] *= np.float32(1e-30)        # squares underflow in fp32, not in fp64
    x[2] *= np.float32(1e30)         # squares overflow in fp32
    x[3] = 0.0
    x[3, 7] = np.float32(1e-42)      # a subnormal alone
    x[4, :] = np.float32(3e38)       # the sum of squares is far above fp32
    x[5, 32:] = 0.0                  # zero blocks beside one that is not
    x[6] *= np.float32(2e-4)         # the size of sqrt(eps)
    for rot, bits in ((0, 4), (32, 8), (128, 4)):
        print("edge rows", rot, bits, flush=True)
        check(torch, x, None, None, bits, rot)
        check(torch, x, None, None, bits, rot, eps=1e-30)
        check(torch, x, np.zeros_like(x), None, bits, rot, eps=1e-40)


def test_nan_and_inf_stay_in_their_row(torch):
    rng = np.random.default_rng(6)
    x, r = draw(rng, 5, 1024, "bf16"), draw(rng, 5, 1024, "bf16")
    clean = bb.rmsnorm_quantize_act(act_to_device(x), residual=act_to_device(r))
    bad = x.copy()
    bad[1, 3] = 0x7FC0   # NaN
    bad[3, 9] = 0x7F80   # inf
    got = bb.rmsnorm_quantize_act(act_to_device(bad), residual=act_to_device(r))
    for a, b in zip(clean, got):
        a, b = host(a), host(b)
        for row in (0, 2, 4):
            assert np.array_equal(a[row], b[row])
    h = f32(host(got[0]))
    assert np.isnan(h[1, 3]) and np.isinf(h[3, 9]) and np.isfinite(np.delete(h[1], 3)).all()


def test_no_rows(torch):
    x = torch.empty(0, 64, device="cuda")
    h, codes, scales = bb.rmsnorm_quantize_act(x, residual=x)
    assert h.shape == (0, 64) and codes.shape == (0, 32) and scales.shape == (0, 2)
    assert bb.dequantize_act(codes, scales).shape == (0, 64)


def test_equals_the_separate_steps(torch):
    """With fp32 input and no residual or weight, the codes are those of the
    quantizer on (x * s)."""
    rng = np.random.default_rng(8)
    x = draw(rng, 33, 2048, "fp32")
    _, v = expected(x, None, None, 1e-6)
    for rot in (0, 32, 64, 128):
        _, codes, scales = bb.rmsnorm_quantize_act(act_to_device(x), rotation=rot)
        vd = act_to_device(v)
        c, s = bb.quantize_act_rot(vd, rot, 4) if rot else bb.quantize_act_unrotated(vd, 4)
        assert torch.equal(codes, c) and torch.equal(scales, s)


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rot", [0, 32, 64, 128])
def test_decode(torch, rot, bits, out):
    for m, k, pad in ((1, 128, 0), (5, 640, 0), (37, 1152, 12), (2, 66048, 4), (700, 384, 0)):
        print("decode", rot, bits, out, m, k, flush=True)
        rng = np.random.default_rng(m + k + rot + bits)
        x = draw(rng, m, k, "bf16")
        q, d = quantized(f32(x), bits, rot)
        codes = torch.from_numpy(oracle_codes(q, bits)).cuda()
        scales = torch.from_numpy(d).cuda()
        dtype = torch.float32 if out == "fp32" else torch.bfloat16
        wide = torch.full((m, k + pad), 3.0, dtype=dtype, device="cuda")
        y = bb.dequantize_act(codes, scales, bits, rot, y=wide[:, :k])
        v = (q.astype(np.float32).reshape(m, -1, 32) * d[:, :, None]).reshape(m, k)
        ref = v if rot == 0 else oracle.rotate_n_f32(v, rot) if rot > 32 else oracle.rotate_f32(v)
        ref = ref if out == "fp32" else synth.bf16_bits(ref)
        got = host(y)
        # (-0 and 0 may differ: the butterflies' signs of zero are not part of the value)
        same = (got == ref) if out == "fp32" else (f32(got) == f32(ref))
        assert same.all(), np.argwhere(~same)[:5]
        assert (wide[:, k:] == 3.0).all()
        if rot:
            v64 = q.astype(np.float64) * np.repeat(d.astype(np.float64), 32, axis=1)
            ref64 = oracle.rotate_n_f64(v64, rot) if rot > 32 else oracle.rotate_f64(v64)
            mag = np.repeat(np.abs(v64).reshape(m, -1, rot).sum(2) / np.sqrt(rot), rot, axis=1)
            # a rounding of code * scale, one a stage, two of the factor, one of the output
            u = 2.0 ** -24
            lim = 1.01 * (3 + np.log2(rot)) * u * mag + (0.0 if out == "fp32" else 2.0 ** -8) * np.abs(ref64) * 1.01
            assert (np.abs(f32(got) - ref64) <= lim + 1e-40).all()


def test_decode_all_codes(torch):
    """Every 4-bit and 8-bit code value, -8 and -128 included (the quantizers never write them)."""
    q4 = np.tile(np.arange(-8, 8, dtype=np.int8), 4)[None, :]
    codes = torch.from_numpy(oracle.pack_int4(q4)).cuda()
    scales = torch.full((1, 2), 0.5, device="cuda")
    assert np.array_equal(host(bb.dequantize_act(codes, scales, 4, 0)), q4 * np.float32(0.5))
    q8 = np.arange(-128, 128, dtype=np.int16).astype(np.int8)[None, :]
    codes = torch.from_numpy(q8.view(np.uint8)).cuda()
    scales = torch.full((1, 8), 2.0, device="cuda")
    assert np.array_equal(host(bb.dequantize_act(codes, scales, 8, 0)), q8 * np.float32(2.0))


def test_round_trip_error(torch):
    """quantize -> decode gives x back within half a step of its rotated block (64-bit norm bound)."""
    rng = np.random.default_rng(12)
    x = draw(rng, 16, 1024, "fp32")
    for bits in (4, 8):
        codes, scales = bb.quantize_act_h32(act_to_device(x), bits)
        y = host(bb.dequantize_act(codes, scales, bits))
        err = np.linalg.norm((y - x).reshape(16, -1, 32), axis=2)
        lim = host(scales).astype(np.float64) * 0.5 * np.sqrt(32)
        # the rotation keeps norms; fp32 roundings of both rotations are below 2^-20 of the block
        assert (err <= lim * (1 + 1e-5) + 2.0 ** -20 * np.linalg.norm(x.reshape(16, -1, 32), axis=2)).all()

"""Routing of tokens to experts.

Bars: the chosen experts equal a plain 64-bit evaluation (ties to the lowest
index), on random logits, tied ones and masked ones; every weight is the
64-bit weight rounded to fp32, within one more rounding's worth of the 64-bit
exponential's error.
"""
import numpy as np
import pytest

from bit_prefill_gemm_amd import binding as bb
from bit_prefill_gemm_amd import synth

from gpu_util import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    return t


def reference(l, topk, score, bias, groups, kept, pair, renorm, scale):
    """The definition, token by token, in 64 bits."""
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max)).astype(np.float64)
    t, e = l.shape
    ids = np.empty((t, topk), dtype=np.int32)
    weights = np.empty((t, topk))
    for i in range(t):
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                p = 1.0 / (1.0 + np.exp(-l[i]))
            elif np.isneginf(l[i]).all():
                p = np.zeros(e)
            else:
                p = np.exp(l[i] - l[i].max())
                p = p / p.sum()
        if bias is not None:
            key = p + bias.astype(np.float64)
            key = np.where(np.isnan(key), -np.inf, key)
        else:
            key = l[i]
        member = np.arange(e)
        if groups > 1:
            size = e // groups
            by = np.sort((key if bias is not None or not pair else p).reshape(groups, size), axis=1)
            with np.errstate(invalid="ignore"):
                g = by[:, -1] + by[:, -2] if pair else by[:, -1]
            g = np.where(np.isnan(g), -np.inf, g)
            chosen = np.argsort(-g, kind="stable")[:kept]
            member = member[np.isin(member // size, chosen)]
        order = member[np.argsort(-key[member], kind="stable")][:topk]
        ids[i] = order
        w = p[order]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(topk)
        weights[i] = w * np.float64(np.float32(scale))
    return ids, weights


def check(torch, l, topk, score="softmax", bias=None, groups=1, kept=1, pair=True, renorm=True,
          scale=1.0, pad=0, bf16=False):
    t, e = l.shape
    print("route", t, e, topk, score, bias is not None, groups, kept, pair, renorm, bf16, flush=True)
    l = synth.bf16_to_f32(synth.bf16_bits(l)) if bf16 else l.astype(np.float32)
    wide = torch.full((t, e + pad), 50.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    wide[:, :e] = torch.from_numpy(l).cuda()
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    ids, w = bb.moe_route_topk(wide[:, :e], topk, score=score, bias=b, groups=groups, topk_groups=kept,
                               group_score="top2" if pair else "max", renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    ref_ids, ref_w = reference(l, topk, score, None if bias is None else bias.astype(np.float32),
                               groups, kept, pair, renorm, scale)
    got = ids.cpu().numpy().reshape(t, topk)
    bad = np.argwhere((got != ref_ids).any(axis=1))
    assert bad.size == 0, (bad[:3].ravel(), got[bad[0, 0]], ref_ids[bad[0, 0]])
    w = w.cpu().numpy().reshape(t, topk).astype(np.float64)
    # one rounding to fp32 (or to its smallest subnormal) and the 64-bit steps' own few 2^-53
    assert (np.abs(w - ref_w) <= (2.0 ** -24 + 2.0 ** -45) * np.abs(ref_w) + 2.0 ** -149).all()
    return got, w


def logits(rng, t, e, spread=2.0):
    return (spread * rng.standard_normal((t, e))).astype(np.float32)


# one expert; a wave's lanes and one more; every count of experts per lane and its ends
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (9, 63, 8), (2, 64, 64), (3, 65, 6),
                                   (17, 127, 9), (512, 128, 8), (6, 129, 4), (33, 256, 8), (5, 257, 8),
                                   (4, 384, 6), (7, 511, 10), (66, 512, 22), (1, 512, 64)])
def test_shapes(torch, t, e, k, score):
    rng = np.random.default_rng(t + e + k)
    check(torch, logits(rng, t, e), k, score)
    check(torch, logits(rng, t, e), k, score, bias=0.2 * rng.standard_normal(e), renorm=False, scale=2.5)
    check(torch, logits(rng, t, e), k, score, pad=3, bf16=True)


@pytest.mark.parametrize("pair", [True, False])
@pytest.mark.parametrize("e,groups,kept,k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 32, 5, 10), (6, 3, 2, 4),
                                             (512, 64, 8, 9), (40, 5, 5, 40), (126, 7, 1, 18), (128, 2, 1, 1),
                                             (300, 4, 2, 64)])
def test_groups(torch, e, groups, kept, k, pair):
    rng = np.random.default_rng(e + groups + k)
    for score in ("softmax", "sigmoid"):
        check(torch, logits(rng, 65, e), k, score, 0.1 * rng.standard_normal(e), groups, kept, pair)
        check(torch, logits(rng, 9, e), k, score, None, groups, kept, pair, renorm=False, bf16=True, scale=16.0)


def test_groups_of_one(torch):
    rng = np.random.default_rng(2)
    check(torch, logits(rng, 20, 16), 4, "sigmoid", None, 16, 5, False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(torch, score):
    rng = np.random.default_rng(4)
    check(torch, np.zeros((3, 200)), 9, score)
    check(torch, np.zeros((3, 200)), 9, score, bias=np.zeros(200), groups=8, kept=3)
    few = rng.integers(0, 3, (40, 512)).astype(np.float32)
    check(torch, few, 33, score)
    check(torch, few, 33, score, bias=rng.integers(0, 2, 512).astype(np.float32))
    check(torch, few, 16, score, None, 16, 7, True)
    check(torch, few, 16, score, None, 16, 7, False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_logits(torch, score):
    """-inf, NaN and the type's lowest value in masked places; rows that keep fewer than topk
    experts, and none."""
    rng = np.random.default_rng(6)
    low = np.finfo(np.float32).min
    for mask in (-np.inf, np.nan, low):
        l = logits(rng, 12, 96)
        l[0, :] = mask
        l[1, 3:] = mask
        l[2, :-2] = mask
        l[3:, rng.random(96) < 0.7] = mask
        check(torch, l, 8, score)
        check(torch, l, 8, score, renorm=False)
        check(torch, l, 8, score, bias=0.1 * rng.standard_normal(96))
        check(torch, l, 8, score, None, 8, 3, True)
    # rows without an open expert and keys that tie or nearly do
    for e in (40, 70):
        l = np.full((3, e), -np.inf)
        l[2, ::3] = 1.0
        steps = np.float32(0.5) + (np.arange(e) % 5 * 2.0 ** -24).astype(np.float32)
        check(torch, l, 6, score, bias=steps)
        check(torch, l, 6, score, bias=np.zeros(e))
        check(torch, l, 6, score)
        check(torch, l, 4, score, steps, 10, 2, True)
        check(torch, l, 4, score, steps, 5, 3, False)
    # experts that are switched off by their bias, for everybody
    b = np.zeros(96)
    b[rng.random(96) < 0.5] = -np.inf
    check(torch, logits(rng, 12, 96), 8, score, bias=b)
    b[5] = np.nan
    b[6] = np.inf
    got, _ = check(torch, logits(rng, 12, 96), 8, score, bias=b)
    assert (got[:, 0] == 6).all()


def test_infinite_and_far_logits(torch):
    rng = np.random.default_rng(7)
    l = logits(rng, 6, 70)
    l[0, [3, 60]] = np.inf             # the two share the weight
    l[1, 9] = np.finfo(np.float32).max
    l[2] *= 1000.0                     # scores underflow, the order of the logits stays
    l[3] = -1e38
    l[4] = 88.0
    _, w = check(torch, l, 5, "softmax")
    assert (w[0, :2] == 0.5).all()
    check(torch, l, 5, "sigmoid")
    check(torch, l, 5, "softmax", renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_closer_than_fp32_tells(torch, score):
    """Keys that differ by less than fp32's rounding of the scores: the choice is that of 64 bits."""
    rng = np.random.default_rng(8)
    e = 192
    one = logits(rng, 1, e)[0]
    p = 1.0 / (1.0 + np.exp(-one.astype(np.float64)))
    if score == "softmax":
        p = np.exp(one.astype(np.float64) - one.max())
        p = p / p.sum()
    level = (1.0 - p).astype(np.float32)          # every key is 1 within 2^-24
    l = np.tile(one, (6, 1))
    l[3:] = logits(rng, 3, e)
    check(torch, l, 9, score, bias=level)
    check(torch, l, 9, score, level, 8, 3, True)
    check(torch, l, 9, score, level, 8, 3, False)
    steps = (np.arange(e) % 7 * 2.0 ** -24).astype(np.float32)
    check(torch, np.full((3, e), 0.25), 12, score, bias=steps)
    # keys of great size and both signs, whose pairs nearly cancel
    far = np.where(np.arange(e) % 2 == 0, 1e6, -1e6) + np.round(rng.standard_normal(e), 1)
    check(torch, l, 9, score, bias=far)
    check(torch, l, 9, score, far, 48, 5, True)


def test_no_tokens_and_many(torch):
    ids, w = bb.moe_route_topk(torch.empty(0, 8, device="cuda"), 2)
    assert ids.shape == (0,) and w.shape == (0,)
    rng = np.random.default_rng(9)
    check(torch, logits(rng, 5003, 60), 4, "softmax")
    # the most entries: only the first and last tokens are compared
    g = torch.Generator(device="cuda").manual_seed(2)
    l = torch.randn(1 << 17, 16, device="cuda", generator=g)
    ids, w = bb.moe_route_topk(l, 8)
    for part in (slice(0, 100), slice(-100, None)):
        ref_ids, _ = reference(l[part].cpu().numpy(), 8, "softmax", None, 1, 1, True, True, 1.0)
        assert np.array_equal(ids.view(-1, 8)[part].cpu().numpy(), ref_ids)


def test_feeds_the_sort(torch):
    """The ids are what the expert sort takes, and the weights sum to the scale."""
    rng = np.random.default_rng(11)
    l = torch.from_numpy(logits(rng, 300, 40)).cuda()
    ids, w = bb.moe_route_topk(l, 6, scale=3.0)
    off, row_token, slot_of = bb.moe_route_sort(ids, 300, 6, 40)
    assert int(off[-1]) == 1800
    assert torch.equal(torch.bincount(ids.long(), minlength=40).cumsum(0).int(), off[1:])
    assert (w.view(300, 6).double().sum(1) - 3.0).abs().max() < 3.0 * 6 * 2.0 ** -24

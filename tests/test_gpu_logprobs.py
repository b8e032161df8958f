"""token_logprobs against the definition in 64 bits.

With u = 2^-23 (an fp32 rounding, or the hardware's exponential) and d = l - m:
every d carries one rounding and is scaled by log2 e with one more, so e^d is
off by a factor 1 + 2 u |d| + 2 u, S by S u (2 E|d| + 4) with the fp32 sums of a
thread's few values (E: the mean under p), T by u (2 E d^2 + 6 E|d|) S.  Then
log S has u (2 E|d| + 4), log p(t) that and the roundings of d and of itself,
and the entropy log S - T / S the two and its own.
"""
import math

import pytest

from bit_prefill_gemm_amd import binding as bb

from gpu_util import torch_mod

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    return t


def check(torch, logits, tokens, topk):
    lp, ent, ids, top = bb.token_logprobs(logits, tokens, topk=topk)
    l = logits.double()
    rows, vocab = l.shape
    m = l.amax(1, keepdim=True)
    d = l - m
    z = torch.logsumexp(d, 1, keepdim=True)
    logp = d - z
    p = logp.exp()
    finite = torch.where(p > 0, d, 0.0)
    e1, e2 = (p * finite.abs()).sum(1), (p * finite ** 2).sum(1)
    tol_s = U * (2 * e1 + 4)
    h = -(p * torch.where(p > 0, logp, 0.0)).sum(1)
    tol_h = tol_s + U * (2 * e2 + 6 * e1 + e1 * (2 * e1 + 4)) + U * h
    assert ent.shape == (rows,) and ((ent.double() - h).abs() <= tol_h).all(), (
        (ent.double() - h).abs() / tol_h).max()
    if tokens is None:
        assert lp is None
    else:
        safe = tokens.long().clamp(0, vocab - 1)[:, None]
        want = torch.gather(logp, 1, safe)[:, 0]
        tol = tol_s + U * (torch.gather(finite, 1, safe)[:, 0].abs() + want.abs())
        good = torch.where(want == -math.inf, lp.double() == -math.inf,
                           (lp.double() - want).abs() <= tol)
        good = torch.where(tokens < 0, lp == 0, good)
        good = torch.where(tokens >= vocab, torch.isnan(lp), good)
        assert good.all()
    assert ids.shape == (rows, topk) and top.shape == (rows, topk)
    if topk:
        order = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :topk]
        assert torch.equal(ids.long(), order), torch.nonzero(ids.long() != order)[:4]
        want = torch.gather(logp, 1, order)
        tol = tol_s[:, None] + U * (torch.gather(finite, 1, order).abs() + want.abs())
        assert ((want == top.double()) | ((top.double() - want).abs() <= tol)).all()


def make(torch, rows, vocab, dtype, kind, seed, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, vocab + pad, generator=g, device="cuda")
    if kind == "normal":
        x *= 3.0
    elif kind == "peaked":
        x[:, vocab // 3] += 40.0
    elif kind == "flat":
        x *= 1e-3
    elif kind == "large":  # far from zero, differences of many orders
        x = x * 300.0 - 5000.0
    elif kind == "ties":  # few distinct values, both zeros among them
        x = (x * 2).round() / 4
    elif kind == "masked":
        x[torch.rand(x.shape, generator=g, device="cuda") < 0.9] = -math.inf
        x[:, 0] = 0.5
    elif kind == "lowest":  # masks of the type's lowest value
        x[torch.rand(x.shape, generator=g, device="cuda") < 0.5] = torch.finfo(dtype).min
        x[:, vocab // 2] = 0.0
    elif kind == "equal":
        x[:] = -2.5
    elif kind == "rising":  # the largest last: every stretch has larger ones than those before
        x = x * 0.01 + torch.arange(vocab + pad, device="cuda") * 0.01
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    return x.to(dtype)[:, :vocab], tokens


KINDS = ["normal", "peaked", "flat", "large", "ties", "masked", "lowest", "equal", "rising"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab,topk,pad", [
    (1, 1, 1, 0), (1, 2, 2, 0), (3, 31, 5, 1), (5, 64, 64, 0), (2, 65, 3, 3), (300, 100, 20, 0),
    (7, 255, 1, 0), (9, 1000, 20, 8), (1, 8191, 64, 0), (33, 8193, 7, 1), (4, 32768, 0, 0),
    (65, 50001, 20, 0), (1, 131072, 20, 0), (2, 131073, 64, 5), (1, 262144, 5, 0), (260, 33000, 32, 2)])
def test_rows(torch, rows, vocab, topk, pad, dtype, kind):
    logits, tokens = make(torch, rows, vocab, getattr(torch, dtype), kind, rows + vocab, pad)
    check(torch, logits, tokens, topk)


@pytest.mark.parametrize("topk", [0, 1, 2, 3, 8, 16, 31, 33, 63, 64])
@pytest.mark.parametrize("vocab", [64, 777, 20000, 70001])
def test_alternatives(torch, vocab, topk):
    for rows in (1, 40, 600):
        for kind in ("normal", "ties", "rising"):
            logits, tokens = make(torch, rows, vocab, torch.bfloat16, kind, topk, 0)
            check(torch, logits, tokens, topk)


@pytest.mark.parametrize("kind", ["huge", "stretches", "tail"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab", [(3, 900), (5, 32768), (300, 40001), (2, 262144)])
def test_wide_ranges_and_stretches(torch, rows, vocab, dtype, kind):
    """Logits up to half the largest, of both signs; masked stretches between open ones; a
    vocabulary padded with -inf."""
    x, tokens = make(torch, rows, vocab, torch.float32, "normal", vocab)
    at = torch.arange(vocab, device="cuda")
    if kind == "huge":
        by = torch.tensor([1e38, 1e30, 1e7, 1e8, 1e12], device="cuda")
        x *= by.repeat(rows // 5 + 1)[:rows, None]
        x = x.clamp(-1.65e38, 1.65e38)  # log probabilities stay in fp32's range
    elif kind == "stretches":
        x[:, at // 700 % 3 == 1] = -math.inf
        x[:, at // 9000 % 2 == 1] = torch.finfo(torch.float32).min
    else:
        x[:, vocab * 3 // 5:] = -math.inf
    check(torch, x.to(getattr(torch, dtype)), tokens, 9)


def test_many_rows(torch):
    for rows, vocab in ((70001, 33), (4099, 2000)):
        logits, tokens = make(torch, rows, vocab, torch.float32, "normal", 1)
        check(torch, logits, tokens, 5)


def test_token_types_and_padding(torch):
    logits, tokens = make(torch, 12, 4000, torch.float32, "normal", 2)
    tokens[3] = -1
    tokens[4] = -100
    tokens[5] = 4000
    tokens[6] = (1 << 40) + 3
    tokens[7] = -(1 << 40)
    check(torch, logits, tokens, 2)
    tokens[6], tokens[7] = 2 ** 31 - 1, -2 ** 31
    check(torch, logits, tokens.to(torch.int32), 2)
    check(torch, logits, None, 2)


@pytest.mark.parametrize("vocab", [40, 5000, 140000])
def test_rows_without_a_distribution(torch, vocab):
    """NaN, +inf, and nothing but -inf: NaN results, ids of the order in which NaN is -inf; the rows
    beside them as ever."""
    for dtype in (torch.float32, torch.bfloat16):
        logits, tokens = make(torch, 6, vocab, dtype, "normal", 3)
        good = logits.clone()
        logits[1, vocab - 1] = math.nan
        logits[2, 7] = math.inf
        logits[3] = -math.inf
        logits[4] = math.nan
        tokens[1] = -1
        lp, ent, ids, top = bb.token_logprobs(logits, tokens, topk=5)
        assert torch.isnan(ent[1:5]).all() and torch.isnan(lp[2:5]).all() and lp[1] == 0
        assert torch.isnan(top[1:5]).all()
        order = torch.where(torch.isnan(logits), -math.inf, logits.float())
        order = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :5]
        assert torch.equal(ids.long(), order)
        want = bb.token_logprobs(good, tokens, topk=5)
        for a, b in zip((lp, ent, ids, top), want):
            assert torch.equal(a[[0, 5]], b[[0, 5]])


def test_given_outputs_and_streams(torch):
    logits, tokens = make(torch, 50, 3000, torch.bfloat16, "normal", 4)
    want = bb.token_logprobs(logits, tokens, topk=6)
    outs = dict(logprobs=torch.empty(50, device="cuda"), entropy=torch.empty(50, device="cuda"),
                ids=torch.empty(50, 6, dtype=torch.int32, device="cuda"),
                top=torch.empty(50, 6, device="cuda"))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = bb.token_logprobs(logits, tokens, topk=6, stream=st, **outs)
    st.synchronize()
    for a, b, name in zip(got, want, outs):
        assert a is outs[name] and torch.equal(a, b)


def test_repeats_and_graphs(torch):
    """The same bits every time, from two graphs that share nothing but the inputs."""
    for rows, vocab in ((1, 131072), (3, 200000), (90, 5000)):
        logits, tokens = make(torch, rows, vocab, torch.float32, "normal", 5)
        want = bb.token_logprobs(logits, tokens, topk=20)
        torch.cuda.synchronize()
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(bb.token_logprobs(logits, tokens, topk=20))
            graphs.append(g)
        for _ in range(4):
            for g, out in zip(graphs, outs):
                for t in out:
                    t.fill_(0)
                g.replay()
                eager = bb.token_logprobs(logits, tokens, topk=20)
                torch.cuda.synchronize()
                for a, b, c in zip(out, want, eager):
                    assert torch.equal(a, b) and torch.equal(c, b)


def test_logits_past_4_gib(torch):
    rows, vocab = 9000, 131072
    logits = torch.zeros(rows, vocab, dtype=torch.float32, device="cuda")
    at = (torch.arange(rows, device="cuda") * 7919) % vocab
    logits[torch.arange(rows, device="cuda"), at] = 20.0
    lp, ent, ids, top = bb.token_logprobs(logits, at, topk=2)
    assert torch.equal(ids[:, 0].long(), at)
    assert torch.equal(ids[:, 1].long(), (at == 0).long())
    want = -math.log1p((vocab - 1) * math.exp(-20.0))
    assert (lp.double() - want).abs().max() <= U * 30 and torch.equal(lp, top[:, 0])


def test_more_rows_than_a_grid_holds(torch):
    """2^26 waves and some: 2^32 threads, over several launches."""
    rows = (1 << 26) + 5
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.empty(rows, 2, dtype=torch.bfloat16, device="cuda").normal_(0, 3, generator=g)
    tokens = torch.arange(rows, dtype=torch.int32, device="cuda") % 2
    out = bb.token_logprobs(logits, tokens, topk=1)
    for at in (0, (1 << 22) - 100, (1 << 25) - 100, (1 << 26) - 100, rows - 200):
        s = slice(at, at + 200)
        check(torch, logits[s], tokens[s], 1)
        for a, b in zip(out, bb.token_logprobs(logits[s], tokens[s], topk=1)):
            assert torch.equal(a[s], b)


def confident(torch, rows, vocab, dtype, seed, beside):
    """Rows whose largest logit stands 1 to 50 above the next; `beside`: the next is its neighbour
    in memory, and alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * 1.5
    at = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    row = torch.arange(rows, device="cuda")
    gap = 1.0 + 49.0 * torch.rand(rows, generator=g, device="cuda")
    if beside:
        x -= 70.0
        x[row, at ^ 1 if vocab % 2 == 0 else (at + 1) % vocab] = 3.3
        x[row, at] = 3.3 + gap
    else:
        x[row, at] = x.amax(1) + gap
    x += 20.0 * torch.rand(rows, 1, generator=g, device="cuda") - 10.0
    return x.to(dtype), at


@pytest.mark.parametrize("beside", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab,topk", [
    (300, 2, 1), (200, 33, 0), (100, 1000, 3), (64, 4096, 20), (40, 5001, 0), (300, 32000, 2),
    (600, 32000, 1), (1, 131072, 20), (9, 131072, 0), (3, 262144, 5)])
def test_confident_rows(torch, rows, vocab, topk, dtype, beside):
    """Log probabilities and entropies near zero, to their own digits.

    With R the sum of e^d, d = l - m, over all logits but the largest, log S = log1p(R) and H =
    log S + (the sum of |d| e^d) / S.  Steps of v = 2^-24: an e^d carries 2.25 v |d| of its exponent
    (a difference, a product, log2 e) and another v |d| of its rescaled sums, 2 v of the exponential,
    4 v of the sum of 16 and 2 v a time that its sums are rescaled (36 of them at most): v (4 |d| +
    80), and its product with d 5 v more.  From R = 1/16 on (1/32 with a margin) the largest logit's
    own term may be off by 10 v of the sum."""
    v = 2.0 ** -24
    for seed in range(3):
        logits, at = confident(torch, rows, vocab, getattr(torch, dtype), seed + vocab, beside)
        l = logits.double()
        first = torch.argmax(l, 1, keepdim=True)
        m = torch.gather(l, 1, first)
        d = l - m
        e = d.exp().scatter(1, first, 0.0)
        r, t = e.sum(1), (d.abs() * e).sum(1)
        d1 = t / r
        d2 = (d * d * e).sum(1) / torch.where(t > 0, t, 1.0)
        log_s = torch.log1p(r)
        near = torch.where(r > 1 / 32, 10 * v, 0.0)
        tol_s = v * (4 * d1 + 80) * r / (1 + r) + near
        h = log_s + t / (1 + r)
        tol_h = tol_s + v * (4 * d2 + 85 + 4 * d1 + 80) * t / (1 + r) + near * (1 + d1) + v * h
        tokens = torch.where(torch.arange(rows, device="cuda") % 3 == 2, (at + 1) % vocab, at)
        lp, ent, ids, top = bb.token_logprobs(logits, tokens, topk=topk)
        assert (lp <= 0).all() and (top <= 0).all() and (ent >= 0).all()
        assert ((ent.double() - h).abs() <= tol_h).all(), ((ent.double() - h).abs() / tol_h).max()
        for got, token in [(lp, tokens)] + [(top[:, j], ids[:, j].long()) for j in range(topk)]:
            want = torch.gather(d, 1, token[:, None])[:, 0] - log_s
            tol = tol_s + v * want.abs()
            assert ((got.double() - want).abs() <= tol).all(), (
                (got.double() - want).abs() / tol).max()


MASKS = ["-inf", "lowest", "-1e4", "nan"]


def mask_to(torch, x, keep, mask):
    """x with one value (or none) wherever `keep` is not set."""
    value = {"-inf": -math.inf, "lowest": torch.finfo(x.dtype).min, "-1e4": -1e4, "nan": math.nan}[mask]
    return torch.where(keep, x, value)


def check_ids(torch, logits, topk):
    """Ids alone, NaN as -inf: by value, then by lowest id."""
    ids = bb.token_logprobs(logits, None, topk=topk)[2]
    l = torch.where(torch.isnan(logits), -math.inf, logits.float())
    order = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :topk]
    assert torch.equal(ids.long(), order), torch.nonzero(ids.long() != order)[:4]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab", [(30, 70), (20, 1500), (12, 4096), (5, 20000), (2, 131072),
                                        (140, 50001), (520, 33000)])
def test_masks_that_leave_few(torch, rows, vocab, dtype, mask):
    """0, 1, 19, 20, 21 and more open logits with 1, 20 and 64 alternatives, anywhere, first or last."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(getattr(torch, dtype))
    at = torch.arange(vocab, device="cuda")
    many = torch.tensor([1, 19, 20, 21, 0, 63, 64, 65, 200, 1100], device="cuda")
    many = many.repeat(rows // 10 + 1)[:rows, None]
    for where in ("anywhere", "first", "last"):
        if where == "anywhere":
            place = torch.argsort(torch.rand(rows, vocab, generator=g, device="cuda"), dim=1)
        else:
            place = (at if where == "first" else at.flip(0)).expand(rows, vocab)
        masked = mask_to(torch, x, place < many, mask)
        for topk in (1, 20, 64):
            check_ids(torch, masked, topk)
        if mask != "nan":
            tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
            some = many[:, 0] > 0
            check(torch, masked[some], tokens[some], 20)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("vocab", [4000, 32768, 140000])
def test_open_logits_of_a_few_threads(torch, vocab, mask, dtype):
    """Thousands of open logits, all in the first ten of every 64 (or 128) threads' places."""
    each = 4 if dtype == "float32" else 8
    g = torch.Generator(device="cuda").manual_seed(vocab)
    for rows in (3, 600):
        x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(getattr(torch, dtype))
        keep = (torch.arange(vocab, device="cuda") // each % 64 < 10).expand(rows, vocab)
        for topk in (9, 20, 64):
            check_ids(torch, mask_to(torch, x, keep, mask), topk)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab", [(4, 3000), (3, 50000), (200, 40000), (600, 20000)])
def test_many_equal_ones_behind_the_largest(torch, rows, vocab, dtype):
    """Equal logits from somewhere on, 5 to 700 larger ones beside them, smaller ones before."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    for first in (0, vocab // 2, vocab - 1400):
        x = torch.randn(rows, vocab, generator=g, device="cuda") - 50.0
        x[:, first:] = 0.5
        for row in range(rows):
            at = torch.randint(0, vocab, ((5, 18, 25, 700)[row % 4],), generator=g, device="cuda")
            x[row, at] = torch.rand(at.shape, generator=g, device="cuda") + 1.0
        x = x.to(getattr(torch, dtype))
        for topk in (1, 20, 64):
            check_ids(torch, x, topk)


def test_masks_cost_no_scans(torch):
    """Rows that a mask leaves ten logits of, or whose logits are equal, take little longer than
    others: they took 60 times as long where each alternative was a scan of the row."""
    rows, vocab = 1024, 131072
    x = (torch.randn(rows, vocab, device="cuda") * 3).bfloat16()
    keep = torch.zeros(rows, vocab, dtype=torch.bool, device="cuda")
    keep.scatter_(1, torch.randint(0, vocab, (rows, 10), device="cuda"), True)

    def time(logits):
        times = []
        for _ in range(7):
            start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            bb.token_logprobs(logits, topk=20)
            stop.record()
            stop.synchronize()
            times.append(start.elapsed_time(stop))
        return min(times)
    plain = time(x)
    for masked in [mask_to(torch, x, keep, m) for m in MASKS] + [torch.full_like(x, -1.0)]:
        assert time(masked) <= 8 * plain


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab", [(3, 700), (4, 4000), (2, 40000), (300, 20000)])
def test_many_at_the_ends_of_the_order(torch, rows, vocab, dtype):
    """Most logits zero (of both signs), the type's largest, +inf, or its smallest step above zero,
    with a few on either side."""
    dt = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(vocab)
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps  # the smallest subnormal
    for value in (0.0, -0.0, torch.finfo(dt).max, math.inf, tiny, -tiny):
        x = torch.full((rows, vocab), value, dtype=dt, device="cuda")
        if value == 0.0:
            x[:, 1::2] = -value
        for other in (1.0, -1.0, tiny, -tiny, 2 * tiny):
            at = torch.randint(0, vocab, (rows, 9), generator=g, device="cuda")
            x.scatter_(1, at, torch.full((rows, 9), other, dtype=dt, device="cuda"))
        for topk in (1, 20, 64):
            check_ids(torch, x, topk)

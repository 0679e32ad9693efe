"""Attention over the 8-bit cache at the edges of what its entry point takes: caches without a
page in every form, value scales of any size, queries that are no finite numbers."""
import numpy as np
import pytest
import torch

from test_gpu_attn_kv8 import Case, halves, near, w  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("n", [1, 4, 33, 900])
def test_no_pages(w, n):
    """Of a cache without pages nothing is read, in the form that converts it first either."""
    print("CASE attn no pages", n, flush=True)
    c = Case([8100, 5], [n, n], 32, 8, 128, 16, spare=0)
    assert halves(w, c, n) == (n == 900)
    kvt, sc, t, lens, st = c.on_device()
    none, nsc = w.kv8_cache(0, 8, 128, 16)
    assert none.numel() == 0
    for kw in (dict(), dict(causal=False), dict(window=3000)):
        out, lse = w.attn_kv8(c.q, none, nsc, t, lens, st, max_rows=n, want_lse=True, **kw)
        assert (out == 0).all() and (lse == float("-inf")).all()


# forms: few rows in one part, in parts and joined, 32 rows a wavefront, tiles, tiles in few and
# in many parts, tiles over the cache converted first
FORMS = [([40, 3], [1, 1], 4, 1), ([9000, 3], [1, 1], 4, 1), ([200, 3], [5, 3], 8, 2),
         ([200, 3], [40, 1], 8, 2), ([1200, 5], [33, 7], 8, 2), ([9000, 5], [33, 7], 8, 2),
         ([8100, 40], [900, 77], 32, 8)]


def spread(c, rows_of_pages):
    """Value scales of the used pages, times what each sequence's pages are given in turn."""
    for s in range(len(c.lens)):
        used = c.table[s][c.table[s] >= 0]
        for i, f in enumerate(rows_of_pages):
            at = used[i::len(rows_of_pages)]
            c.scales[at, :, 1] = (c.scales[at, :, 1].astype(np.float64) * f).astype(np.float32)


@pytest.mark.parametrize("past,n,hq,hk", FORMS)
@pytest.mark.parametrize("scales", [(0.0, 2.0 ** 45), (2.0 ** 45, 0.0), (2.0 ** -60, 2.0 ** 60, 1.0),
                                    (2.0 ** 120, 2.0 ** -120, 0.0), (2.0 ** -130, 1.0),
                                    (2.0 ** 120,), (2.0 ** -125,), (0.0,), (1.0, 1.0, 0.0)])
def test_value_scales_of_any_size(w, past, n, hq, hk, scales):
    """A token weighs the same in the softmax's sum whatever its page's value scale is: pages
    of zeros, scales far apart, at both ends of what binary32 holds."""
    print("CASE attn value scales", past, n, hq, hk, scales, flush=True)
    c = Case(past, n, hq, hk, 32 if n[0] == 900 else 64, 16, seed=len(scales))
    if n[0] == 900:
        assert halves(w, c, 900)
    spread(c, scales)
    used = c.table[c.table >= 0]
    assert np.isfinite(c.scales[used]).all()
    for kw in (dict(), dict(window=70)) if n[0] < 100 else (dict(),):
        out, lse = c.check(w, max_rows=max(n), **kw)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_equal_scores_beside_zeros(w):
    """Sixteen tokens of zeros and sixteen ones at equal scores: half of one's value, ln 32."""
    c = Case([31], [1], 4, 1, 64, 16)
    c.q.zero_()
    c.codes[1] = 1
    for big in (2.0 ** 29, 2.0 ** 40, 2.0 ** 127):
        c.scales[c.table[0, :2], 0, 1] = 0.0, big
        out, lse = c.run(w)
        assert torch.equal(out, torch.full_like(out, big / 2))
        assert (lse - np.log(32)).abs().max() < 1e-6


def test_many_tokens_of_zeros(w):
    """Enough of them that their number times a factor for their scale would leave binary32."""
    c = Case([150000, 7], [1, 1], 1, 1, 32, 128)
    c.q.zero_()
    c.scales[c.table[0], :, 1] = 0.0
    out, lse = c.run(w)
    assert (out[0] == 0).all() and abs(lse[0, 0].item() - np.log(150001)) < 1e-5


@pytest.mark.parametrize("past,n,hq,hk", FORMS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_queries_that_are_not_finite(w, past, n, hq, hk, bad):
    """NaN in the rows that hold one and see a token, whatever the signs of what they see; a row
    that sees nothing gives 0 and -inf, and the others are as they were."""
    print("CASE attn queries", past, n, hq, hk, bad, flush=True)
    c = Case(past, n, hq, hk, 32 if n[0] == 900 else 64, 16)
    if past[0] == 200:
        c.lens[0] = n[0] - 1                                # its first row sees nothing
    if past[0] == 1200:
        c.table[0] = -1                                     # no row of it does
    c.codes[0] = np.where(c.codes[0] == 0, 1, c.codes[0])   # no 0 that an infinity makes NaN
    o, l, eo, el = c.want(max_rows=max(n))
    hit = torch.zeros(l.shape, dtype=torch.bool, device="cuda")
    for row, head in ((0, 0), (0, hq - 1), (n[0] // 2, 1), (n[0], 2)):
        if row < len(c.q):
            c.q[row, head, 5] = bad
            hit[row, head] = l[row, head] > float("-inf")
    out, lse = c.run(w, max_rows=max(n))
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    near(out[~hit], lse[~hit], o[~hit], l[~hit], eo[~hit], el[~hit])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
def test_one_token_of_either_sign(w, bad):
    """One sign decides in the first row of a prompt: a score of -inf is NaN too."""
    for sign in (1, -1):
        c = Case([0], [3], 4, 1, 64, 16)
        c.codes[0] = sign * 3
        c.q[0, 1, 7] = bad
        out, lse = c.run(w, scale=sign * 0.1)
        assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
        assert torch.isfinite(out[1:]).all() and torch.isfinite(lse[0, 2:]).all()
        out, lse = c.run(w)
        assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])


@pytest.mark.parametrize("past,n,hq,hk", FORMS)
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf")])
def test_scales_of_scores_that_are_not_finite(w, past, n, hq, hk, scale):
    """NaN in every row that sees a token, 0 and -inf in the others."""
    print("CASE attn scale", past, n, hq, hk, scale, flush=True)
    c = Case(past, n, hq, hk, 32 if n[0] == 900 else 64, 16)
    c.lens[1] = n[1] - 1
    c.q[0] = 0.0
    out, lse = c.run(w, max_rows=max(n), scale=scale)
    none = n[0]                                             # that row sees nothing
    assert (lse[none] == float("-inf")).all() and (out[none] == 0).all()
    some = torch.arange(len(c.q), device="cuda") != none
    assert torch.isnan(lse[some]).all() and torch.isnan(out[some]).all()


@pytest.mark.parametrize("past,n,hq,hk", FORMS)
@pytest.mark.parametrize("size,scale", [(2.0 ** -115, 2.0 ** 112), (2.0 ** -125, 2.0 ** 122),
                                        (2.0 ** -131, 2.0 ** 126)])
def test_tiny_queries(w, past, n, hq, hk, size, scale):
    """Down to subnormal bf16, with a scale that brings the scores back: no element loses bits
    (all are multiples of 2^-133), the smallest of a row neither."""
    print("CASE attn tiny queries", past, n, hq, hk, size, flush=True)
    c = Case(past, n, hq, hk, 32 if n[0] == 900 else 64, 16, sharp=2.0)
    c.q[..., ::2] *= 2.0 ** -10
    c.q = (c.q.float() * size).to(BF)
    assert (c.q != 0).any()
    c.check(w, max_rows=max(n), scale=scale)
    c.q[..., 1::2] = 0                                      # what a row's largest would hide
    c.check(w, max_rows=max(n), scale=scale)


@pytest.mark.parametrize("dim,hq,rows", [(32, 8, 1), (96, 5, 1), (128, 4, 1), (128, 8, 2), (192, 8, 4), (256, 4, 3)])
@pytest.mark.parametrize("past", [3, 4000])
def test_weights_of_few_rows_keep_22_bits(w, dim, hq, rows, past):
    """Up to 16 packed rows (64 past 128 elements a head) the weights enter the sum over the values
    with 22 bits: out is the right one rounded to bf16, but for what the other steps may be off by.
    Few tokens of large weight, each with a query of one element, so that those are small:
      score   one product: 4 u (|s| + |lse| + 128) for the factors and the exponent's sum (as in
              kv8_util.attention, whose first term is the sum of dim products)
      weight  exp2 2^-22, two halves 2^-22, or below 2^-14 of a reference that is at most a 16th of
              the largest weight 2^-25 of that
    A half alone may be off by 2^-12."""
    print("CASE attn 22 bits", dim, hq, rows, past, flush=True)
    c = Case([past] * 40, [rows] * 40, hq, 1, dim, 16, seed=dim + past)
    c.scales[:, :, 0] *= 16.0
    g = torch.Generator(device="cuda").manual_seed(past)
    at = torch.randint(0, dim, (len(c.q), hq, 1), generator=g, device="cuda")
    c.q = torch.zeros_like(c.q).scatter_(2, at, torch.randn(at.shape, generator=g, device="cuda").to(BF) + 1)
    if past > 100:                                          # few tokens with a weight among many
        c.codes[0, :, :, 1:] = np.clip(c.codes[0, :, :, 1:], -20, 20)
    out, lse = c.run(w, max_rows=rows, scale=0.25)
    u = 2.0 ** -24
    for s in range(40):
        n = past + rows
        page = torch.from_numpy(c.table[s][np.arange(n) // 16]).cuda().long()
        slot = torch.arange(n, device="cuda") % 16
        k, v = (torch.from_numpy(c.codes[i]).cuda()[page, 0, slot].double() *
                torch.from_numpy(c.scales).cuda()[page, 0, i, None].double() for i in range(2))
        sv = torch.from_numpy(c.scales).cuda()[page, 0, 1].double()
        for i in range(rows):
            r, m = s * rows + i, past + i + 1               # tokens seen
            score = 0.25 * torch.matmul(c.q[r].double(), k[:m].T.contiguous())
            l = torch.logsumexp(score, 1, keepdim=True)
            p = torch.exp(score - l)
            o, a = torch.matmul(p, v[:m]), torch.matmul(p, v[:m].abs())
            ds = 4 * u * (score.abs().amax(1, keepdim=True) + l.abs() + 128)
            unit = (p * sv[:m]).amax(1, keepdim=True)
            bound = (2 * ds + 2.0 ** -21 + 2.0 ** -21 + 2 * u * (m + 64)) * a + m * 2.0 ** -29 * 127 * unit
            half = torch.exp2(torch.floor(torch.log2(o.abs().clamp_min(2.0 ** -120))) - 8)   # of a step
            off = (out[r].double() - o).abs()
            assert (off <= half + bound * (1 + 2.0 ** -7)).all(), (off / (half + bound)).max().item()

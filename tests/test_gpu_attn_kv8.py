"""Attention over the 8-bit cache against the formula in 64 bits, within what the kernel's
roundings can add up to (kv8_util.attention)."""
import numpy as np
import pytest
import torch

import kv8_util as kv

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def w():
    from w4a8_quantized_gemm_quantize_amd import binding
    torch.cuda.init()
    return binding


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Sequences of `past + n` tokens in a cache whose other bytes are rubbish, its unused
    scales NaN; `sharp` scales the queries."""

    def __init__(self, past, n, hq, hk, dim, page, seed=0, sharp=1.0, spare=3, blocks=None, device="cuda"):
        rng = np.random.default_rng(seed)
        self.lens = np.array(past, np.int64) + np.array(n)
        self.starts, self.n = kv.starts_of(n), n
        need = int(sum(-(-max(x, 0) // page) for x in self.lens))
        pages = need + spare
        self.table = kv.make_table(self.lens, page, pages, rng, blocks)
        self.codes = np.clip(np.rint(rng.standard_normal((2, pages, hk, page, dim)) * 35), -127,
                             127).astype(np.int8)
        self.scales = (rng.uniform(0.5, 2.0, (pages, hk, 2)) / 35).astype(np.float32)
        self.scales[~np.isin(np.arange(pages), self.table)] = np.nan
        self.q = dev((rng.standard_normal((int(self.starts[-1]), hq, dim)) * sharp)
                     .astype(np.float32)).to(BF)
        self.lens = self.lens.astype(np.int32)
        self.sizes = hq, hk, dim, page

    def on_device(self):
        return (dev(kv.pack(self.codes)), dev(self.scales), dev(self.table), dev(self.lens),
                dev(self.starts))

    def run(self, w, null_start=False, **kw):
        kvt, sc, t, lens, st = self.on_device()
        return w.attn_kv8(self.q, kvt, sc, t, lens, None if null_start else st, want_lse=True, **kw)

    def want(self, **kw):
        return kv.attention(self.q, dev(self.codes), dev(self.scales), self.table,
                            self.lens.tolist(), self.starts, **kw)

    def check(self, w, null_start=False, max_rows=None, **kw):
        out, lse = self.run(w, null_start=null_start, max_rows=max_rows, **kw)
        near(out, lse, *self.want(**kw))
        return out, lse


def near(out, lse, o, l, eo, el):
    half = torch.finfo(BF).eps / 2
    room = eo * (1 + half) + half * o.abs() + 2.0 ** -126
    off = (out.double() - o).abs()
    assert (off <= room).all(), f"out: {(off / room).max().item()} of what it may be"
    empty = l == float("-inf")
    assert torch.equal(lse == float("-inf"), empty)
    off = (lse.double() - l).abs()[~empty]
    assert (off <= el[~empty]).all(), f"lse: {(off / el[~empty]).max().item()} of what it may be"


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hk", [(8, 1), (6, 2)])
def test_ragged(w, dim, page, hq, hk):
    print("CASE attn ragged", dim, page, hq, hk, flush=True)
    Case([0, 3, 0, 100, 17, 31, 250], [1, 5, 40, 0, 16, 1, 2], hq, hk, dim, page).check(w)


@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 1), (16, 1), (14, 2), (64, 1), (20, 1), (17, 1), (32, 4)])
@pytest.mark.parametrize("lens", [[1], [0], [15, 16, 17, 31, 32, 33, 63, 64, 65], [700, 1, 0, 2000]])
def test_single_tokens(w, hq, hk, lens):
    print("CASE attn single", hq, hk, lens, flush=True)
    c = Case([x - 1 for x in lens], [1] * len(lens), hq, hk, 64, 16)
    a = c.check(w, null_start=True)
    b = c.run(w)
    c2 = c.run(w, max_rows=1)
    assert torch.equal(a[0], c2[0]) and torch.equal(a[1], c2[1])
    near(*b, *c.want())


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("hq,hk", [(8, 1), (16, 2), (14, 2), (5, 1)])
@pytest.mark.parametrize("kw", [dict(), dict(window=20), dict(causal=False)])
def test_few_rows(w, dim, hq, hk, kw):
    """A few rows a sequence: 10 to 40 packed rows, one or two tiles of them."""
    print("CASE attn few rows", dim, hq, hk, kw, flush=True)
    c = Case([0, 100, 0, 33, 700], [5, 2, 1, 3, 5], hq, hk, dim, 16, seed=dim, sharp=2.0)
    c.scales[c.table[4, :8], :, 1] *= np.float32(2.0 ** 10)
    c.table[1, 2] = -1
    c.check(w, max_rows=5, **kw)


@pytest.mark.parametrize("window", [1, 2, 16, 33, 1000])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(w, window, causal):
    Case([0, 90, 300, 5], [70, 1, 33, 5], 4, 2, 64, 32, seed=window).check(w, window=window,
                                                                       causal=causal)


@pytest.mark.parametrize("n", [1, 4, 60])
def test_behind_the_window(w, n):
    """Pages that slid out of the window may be gone or hold anything."""
    c = Case([500, 330], [n, n], 4, 2, 64, 16, seed=n)
    for s, length in enumerate(c.lens):
        out = max(0, int(length) - n - 100 + 1) // 16           # wholly before every row's window
        for b in range(out):
            c.scales[c.table[s, b]] = [np.nan, np.inf, -np.inf, 0.0][b % 4]
        c.table[s, 0:out:5] = -1
    c.check(w, window=100, max_rows=n)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -1.0])
@pytest.mark.parametrize("part", [0, 1])
@pytest.mark.parametrize("past,n", [(300, 1), (30000, 3), (300, 10), (300, 90), (6000, 90),
                                    (8100, 900)])
def test_scales_that_are_no_numbers(w, past, n, part, bad):
    """Rows that see such a page say so, the others are as they were."""
    print("CASE attn scales", past, n, part, bad, flush=True)
    c = Case([past, 200], [n, n], 8, 2, 32, 16, seed=n)
    if past == 8100:
        c = Case([past, 200], [n, n], 32, 8, 32, 16, seed=n)
        assert halves(w, c, n)
    o, l, eo, el = c.want()
    at = past + n // 2                                        # in the middle of the rows
    c.scales[c.table[0, at // 16], 1, part] = bad
    out, lse = c.run(w, max_rows=n)
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    hit[max(0, at // 16 * 16 - past):n, 4:8] = True
    assert hit.any() and torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    near(out[~hit], lse[~hit], o[~hit], l[~hit], eo[~hit], el[~hit])


def test_queries_that_are_no_numbers(w):
    """In their own rows only."""
    c = Case([50, 400], [3, 90], 8, 2, 64, 16)
    o, l, eo, el = c.want()
    c.q[1, 2, 5] = c.q[40, 7, 63] = float("nan")
    out, lse = c.run(w, max_rows=90)
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    hit[1, 2] = hit[40, 7] = True
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    near(out[~hit], lse[~hit], o[~hit], l[~hit], eo[~hit], el[~hit])


def test_windows_that_32_bits_do_not_hold(w):
    c = Case([50], [3], 8, 2, 64, 16)
    for window in (-1, (1 << 30) + 1, (1 << 32) + 5, -(1 << 32) + 5):
        with pytest.raises(w.W4A8Error):
            c.run(w, window=window)
    c.check(w, window=1 << 30)


def test_not_causal(w):
    Case([0, 90, 300], [70, 1, 33], 6, 2, 128, 16).check(w, causal=False)


@pytest.mark.parametrize("sharp", [0.0, 0.1, 8.0, 60.0])
def test_flat_and_sharp(w, sharp):
    """From equal weights to one token that takes all, with rows that see more and more."""
    Case([0, 2000], [130, 3], 8, 2, 128, 16, sharp=sharp).check(w)


@pytest.mark.parametrize("rows", [1, 3, 16, 100])
def test_long(w, rows):
    """Few rows over a long axis: split over workgroups and joined."""
    c = Case([30011, 12], [rows, rows], 8, 2, 128, 64)
    need = w.attn_kv8_workspace_bytes(2 * rows, 2, True, rows, c.table.shape[1], 8, 2, 128, 64)
    assert need > 0 or rows > 3
    c.check(w, max_rows=rows)


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("past,few", [(1200, True), (3000, False)])
def test_tiles_in_parts(w, dim, past, few):
    """Tiles over few and over many parts of the tokens, which two kernels join: a sequence
    shorter than a part, one without rows, and one row that sees nothing."""
    if dim == 32:
        past *= 2                                             # parts of it are longer
    print("CASE attn parts", dim, past, flush=True)
    c = Case([past, 5, 40, 0], [33, 7, 0, 90], 8, 2, dim, 16, seed=dim)
    c.lens[1] = 6                                             # seven rows, six tokens
    need = w.attn_kv8_workspace_bytes(130, 4, True, 90, c.table.shape[1], 8, 2, dim, 16)
    tiles = 130 * 4 // 128 + 4
    parts = need // (tiles * 2 * 128 * (dim + 4) * 4)
    assert 1 < parts <= 8 if few else parts > 8
    out, lse = c.check(w, max_rows=90)
    assert (lse[33] == float("-inf")).all() and (out[33] == 0).all()


@pytest.mark.parametrize("dim,rows", [(64, 700), (128, 500), (256, 300), (96, 333)])
def test_prompts(w, dim, rows):
    Case([0, 0, 1000], [rows, 77, rows // 2], 8, 2, dim, 16).check(w, max_rows=rows)


def halves(w, c, max_rows):
    """Whether the call takes the form that converts the cache first (by its workspace)."""
    hq, hk, dim, page = c.sizes
    blocks = c.table.shape[1]
    need = w.attn_kv8_workspace_bytes(len(c.q), len(c.n), True, max_rows, blocks, hq, hk, dim, page)
    return need >= len(c.n) * hk * ((blocks * page + 63) // 64) * 64 * dim * 4


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_long_prompts(w, dim):
    """Many tiles over many tokens: from the cache converted once."""
    print("CASE attn halves", dim, flush=True)
    c = Case([8100, 0, 2500], [900, 1, 77], 32, 8, dim, [16, 32, 64, 128][dim // 32 % 4])
    assert halves(w, c, 900) and not halves(w, Case([0], [200], 32, 8, dim, 16), 200)
    c.check(w, max_rows=900)


@pytest.mark.parametrize("kw", [dict(window=3000), dict(causal=False, window=4000)])
def test_long_prompts_in_windows(w, kw):
    """Windows of many tiles: the halves of what they see."""
    c = Case([8100, 5], [1800, 77], 64, 16, 32, 16, seed=6)
    assert halves(w, c, 1800)
    # behind the window of every row: the first sees tokens from 8101 - window on
    c.scales[c.table[0, :(8101 - kw["window"]) // 16]] = np.nan
    c.check(w, max_rows=1800, **kw)


@pytest.mark.parametrize("kw", [dict(window=1000), dict(window=30), dict(causal=False),
                                dict(causal=False, window=2000)])
def test_long_prompts_seen_otherwise(w, kw):
    c = Case([8100, 2500], [900, 77], 32, 8, 64, 16, seed=5)
    assert halves(w, c, 900)
    c.table[0, 7:9] = -1                                      # no pages
    c.table[0, 200] = len(c.scales)
    c.scales[c.table[0, 100:120], :, 1] *= np.float32(2.0 ** 12)
    c.scales[c.table[0, 150], :, 1] = 0
    c.check(w, max_rows=900, **kw)


def test_long_prompts_by_graph(w):
    """Captured, with other pages and lengths at each replay; the space between is reused."""
    c = Case([8100, 2500], [900, 77], 32, 8, 64, 16, seed=6)
    kvt, sc, t, lens, st = c.on_device()
    need = w.attn_kv8_workspace_bytes(len(c.q), 2, True, 900, t.shape[1], 32, 8, 64, 16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")     # halves are NaN
    l, tt = lens.clone(), t.clone()
    out, lse = torch.empty_like(c.q), torch.empty((len(c.q), 32), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.attn_kv8(c.q, kvt, sc, tt, l, st, max_rows=900, out=out, lse=lse, workspace=ws)
    for i in range(3):
        l.copy_(lens - 450 * i)
        tt[0, 5:50] = t[0, 5:50].flip(0) if i == 1 else t[0, 5:50]
        graph.replay()
        a = w.attn_kv8(c.q, kvt, sc, tt, l, st, max_rows=900, want_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, a[0]) and torch.equal(lse, a[1])
    c.lens = (lens - 900).cpu().numpy()
    near(out, lse, *c.want(max_rows=900))


def test_scales_far_apart(w):
    """Pages of values 2^40 apart, zero pages, the largest scale on a page of no weight."""
    c = Case([0, 200], [200, 3], 4, 1, 64, 16, seed=3, sharp=3.0)
    used = c.table[c.table >= 0]
    for i, f in enumerate([2.0 ** -40, 0.0, 1.0, 2.0 ** 20]):
        c.scales[used[i::5], :, 1] *= np.float32(f)
    c.codes[1][c.scales[..., 1] == 0] = 0
    c.scales[used[3], :, 0] = 0.0
    c.check(w)
    c.scales[used, :, 1] = 0
    c.codes[1] = 0
    out, lse = c.check(w)
    assert (out == 0).all()


@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** -90, 2.0 ** 120])
def test_query_sizes(w, size):
    """Queries far from 1 with a scale that brings the scores back."""
    c = Case([0, 40], [33, 1], 4, 2, 64, 16)
    c.q = (c.q.float() * size).to(BF)
    c.check(w, scale=0.125 / size)


def test_query_elements_far_apart(w):
    c = Case([0, 40], [33, 1], 4, 2, 64, 16)
    c.q[..., ::3] *= 2.0 ** -30
    c.q[..., 1] *= 2.0 ** 6
    c.check(w)


def test_zero_queries_and_negative_scale(w):
    c = Case([0, 40], [33, 1], 4, 2, 64, 16)
    c.q[3:9] = 0
    c.check(w, scale=-0.2)
    c.check(w, scale=0.0)


def test_pages_that_are_none(w):
    c = Case([0, 100, 60], [50, 3, 30], 4, 2, 64, 16)
    c.table[0, 1] = -1
    c.table[1, 0] = len(c.scales)
    c.table[1, 6] = -7
    c.table[2, :] = -1
    out, lse = c.check(w)
    assert (lse[53:] == float("-inf")).all() and (out[53:] == 0).all()
    c.table[:] = -1
    out, lse = c.check(w)
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_rows_that_see_nothing(w):
    """More rows than tokens, no tokens at all, a table that ends early."""
    c = Case([0, 100], [50, 3], 4, 2, 64, 16)
    c.lens[0] = 20
    out, lse = c.check(w)
    assert (lse[:30] == float("-inf")).all() and (lse[30:50] > float("-inf")).all()
    c.lens[:] = [0, -4]
    out, lse = c.check(w)
    assert (out == 0).all()
    c = Case([0, 100], [50, 3], 4, 2, 64, 16)
    c.table = np.ascontiguousarray(c.table[:, :2])
    c.check(w)


def test_rows_left_alone(w):
    """Behind the last sequence, before the first, past max_rows."""
    c = Case([5, 100, 0], [9, 3, 20], 4, 2, 64, 16)
    kvt, sc, t, lens, st = c.on_device()
    q = torch.zeros((40, 4, 64), dtype=BF, device="cuda")
    q[2:34] = c.q
    out = torch.full((40, 4, 64), 7.0, dtype=BF, device="cuda")
    lse = torch.full((40, 4), 7.0, device="cuda")
    w.attn_kv8(q, kvt, sc, t, lens, st + 2, max_rows=8, out=out, lse=lse)
    o, l, eo, el = c.want(max_rows=8)
    some = ~torch.isnan(l[:, 0])
    near(out[2:34][some], lse[2:34][some], o[some], l[some], eo[some], el[some])
    left = torch.cat([torch.tensor([True] * 2, device="cuda"), ~some,
                      torch.tensor([True] * 6, device="cuda")])
    assert int(left.sum()) == 8 + 1 + 12
    assert (out[left] == 7).all() and (lse[left] == 7).all()


def test_strides(w):
    c = Case([0, 40, 7], [20, 1, 5], 6, 2, 96, 32)
    kvt, sc, t, lens, st = c.on_device()
    want = c.run(w)
    wide = torch.zeros((26, 10 * 96 + 8), dtype=BF, device="cuda")
    q = wide[:, 96:7 * 96].view(26, 6, 96)
    q.copy_(c.q)
    out = torch.full((26, 8, 96), 7.0, dtype=BF, device="cuda")
    tt = torch.full((5, 9), -1, dtype=torch.int32, device="cuda")
    tt[1:4, 3:3 + t.shape[1]] = t
    tt = tt[1:4, 3:3 + t.shape[1]]
    got = w.attn_kv8(q, kvt, sc, tt, lens, st, out=out[:, :6])
    assert torch.equal(got, want[0]) and (out[:, 6:] == 7).all()


def test_same_bits_every_time(w):
    c = Case([3000, 10], [40, 40], 8, 2, 128, 16)
    a, b = c.run(w), c.run(w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_past_4_gib(w):
    heads, dim, page = 8, 256, 128
    c = Case([150], [3], 16, heads, dim, page)
    kvt, sc, t, lens, st = c.on_device()
    want = c.run(w)
    pages = (5 << 30) // (heads * 2 * page * dim) + 8
    big = torch.empty((pages, heads, 2, page, dim), dtype=torch.uint8, device="cuda")
    n = kvt.shape[0]
    big[-n:] = kvt
    bsc = torch.zeros((pages, heads, 2), device="cuda")
    bsc[-n:] = sc
    t = torch.where(t >= 0, t + (pages - n), t)
    got = w.attn_kv8(c.q, big, bsc, t, lens, st, want_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_streams_workspaces_graphs(w):
    """On another stream; a shared workspace; captured, with new lengths and tokens at each
    replay."""
    c = Case([2500, 800, 10], [1, 1, 1], 8, 2, 128, 16, blocks=200)
    kvt, sc, t, lens, st = c.on_device()
    want = c.run(w, null_start=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = w.attn_kv8(c.q, kvt, sc, t, lens, want_lse=True, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    need = w.attn_kv8_workspace_bytes(3, 3, False, 1, 200, 8, 2, 128, 16)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    with pytest.raises(w.W4A8Error):
        w.attn_kv8(c.q, kvt, sc, t, lens, workspace=ws[:need - 1])
    q, l = c.q.clone(), lens.clone()
    out, lse = torch.empty_like(q), torch.empty((3, 8), device="cuda")
    out2, l2 = torch.empty_like(q), lens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.attn_kv8(q, kvt, sc, t, l, out=out, lse=lse, workspace=ws)
        w.attn_kv8(q, kvt, sc, t, l2, out=out2, window=100, workspace=ws)
    for i in range(4):
        g = torch.Generator(device="cuda").manual_seed(i)
        q.copy_(torch.randn(q.shape, generator=g, device="cuda").to(BF))
        l.copy_(lens - i * torch.tensor([400, 100, 3], device="cuda", dtype=torch.int32))
        graph.replay()
        a = w.attn_kv8(q, kvt, sc, t, l, want_lse=True)
        b = w.attn_kv8(q, kvt, sc, t, l2, window=100)
        torch.cuda.synchronize()
        assert torch.equal(out, a[0]) and torch.equal(lse, a[1]) and torch.equal(out2, b)


def test_graphs_that_share_a_workspace(w):
    """Two graphs, replayed in turn on one stream, with eager calls between them."""
    c = Case([2500, 800], [2, 2], 8, 2, 128, 16, seed=3)
    kvt, sc, t, lens, st = c.on_device()
    need = w.attn_kv8_workspace_bytes(4, 2, True, 2, t.shape[1], 8, 2, 128, 16)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(c.q) for _ in range(2)], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w.attn_kv8(c.q, kvt, sc, t, lens, st, max_rows=2, window=700 * i, out=outs[i], workspace=ws)
        graphs.append(g)
    want = [w.attn_kv8(c.q, kvt, sc, t, lens, st, max_rows=2, window=700 * i) for i in range(2)]
    for _ in range(3):
        for o in outs:
            o.zero_()
        graphs[0].replay()
        graphs[1].replay()
        eager = w.attn_kv8(c.q, kvt, sc, t, lens, st, max_rows=2, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
        assert torch.equal(eager, want[0])


def test_two_streams_at_once(w):
    c, d = Case([6000], [3], 8, 2, 128, 16, seed=4), Case([300], [200], 8, 2, 64, 32, seed=5)
    want = c.run(w), d.run(w)
    args = [(x.q, *x.on_device()) for x in (c, d)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            got[i].append(w.attn_kv8(*args[i], want_lse=True, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_empty(w):
    c = Case([10], [4], 4, 2, 64, 16)
    kvt, sc, t, lens, st = c.on_device()
    none = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    assert w.attn_kv8(none, kvt, sc, t[:0], lens[:0]).shape == (0, 4, 64)
    assert w.attn_kv8(none, kvt, sc, t, lens, st * 0).shape == (0, 4, 64)
    kv0, sc0 = w.kv8_cache(0, 2, 64, 16)
    out, lse = w.attn_kv8(c.q, kv0, sc0, t, lens, st, want_lse=True)
    assert (out == 0).all() and (lse == float("-inf")).all()
    assert (w.attn_kv8(c.q, kvt, sc, t[:, :0], lens, st) == 0).all()


def test_refusals(w):
    c = Case([10], [4], 4, 2, 64, 16)
    kvt, sc, t, lens, st = c.on_device()
    good = dict(q=c.q, kv=kvt, kv_scale=sc, block_table=t, lens=lens, row_start=st)
    for bad in (dict(q=c.q.float()), dict(q=c.q[..., :32]), dict(q=c.q[:, :3]), dict(q=c.q[0]),
                dict(row_start=st.long()), dict(row_start=None), dict(kv_scale=sc[:1]),
                dict(block_table=t[0]), dict(max_rows=0), dict(window=-1),
                dict(out=c.q[:3]), dict(out=c.q.float()), dict(lse=sc[:1]),
                dict(lse=torch.zeros(16, dtype=torch.float64, device="cuda"))):
        with pytest.raises((ValueError, w.W4A8Error)):
            w.attn_kv8(**{**good, **bad})

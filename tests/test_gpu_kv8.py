"""The paged 8-bit cache: writes against the binary32 steps in numpy, bit for bit (codes,
scales, and every byte that is not theirs), and reading back."""
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


class Cache:
    """The cache on the device and its model, both full of the same rubbish."""

    def __init__(self, w, pages, heads, dim, page, seed):
        rng = np.random.default_rng(seed)
        self.w = w
        self.codes = rng.integers(-127, 128, (2, pages, heads, page, dim)).astype(np.int8)
        self.scales = rng.uniform(0.001, 0.1, (pages, heads, 2)).astype(np.float32)
        self.kv, self.sc = dev(kv.pack(self.codes)), dev(self.scales)

    def write(self, k, v, table, lens, starts, null_start=False, **kw):
        self.w.kv8_write(k, v, self.kv, self.sc, dev(table), dev(np.asarray(lens, np.int32)),
                         None if null_start else dev(starts), **kw)
        kv.write(self.codes, self.scales, table, lens, starts,
                 [x.float().cpu().numpy() for x in (k, v)])

    def same(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.sc.cpu().numpy().view(np.int32), self.scales.view(np.int32))
        got = kv.unpack(self.kv.cpu().numpy())
        assert np.array_equal(got, self.codes), np.argwhere(got != self.codes)[:5]


def rows(n, heads, dim, dt, seed, spread=1.0):
    """k and v as columns of one projection's rows, rows of different sizes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, 2 * heads * dim + 8), generator=g, device="cuda")
    x = (x * torch.exp(spread * torch.randn((n, 1), generator=g, device="cuda"))).to(dt)
    return (x[:, :heads * dim].view(n, heads, dim),
            x[:, heads * dim:2 * heads * dim].view(n, heads, dim))


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dt", [BF, F])
def test_prompts_and_what_follows(w, dim, page, dt):
    """Ragged prompts, then more rows for each, then a few single tokens."""
    print("CASE kv8 write", dim, page, dt, flush=True)
    rng = np.random.default_rng(dim + page)
    heads = 3
    n1, n2 = [1, 40, 0, 129, 16, 15], [5, 0, 3, 70, 16, 1]
    lens = np.array(n1)
    table = kv.make_table(lens + np.array(n2) + 4, page, 64, rng)
    c = Cache(w, 64, heads, dim, page, 1)
    st = kv.starts_of(n1)
    c.write(*rows(int(st[-1]) + 2, heads, dim, dt, 2), table, lens, st)
    c.same()
    st = kv.starts_of(n2)
    lens = lens + np.array(n2)
    c.write(*rows(int(st[-1]), heads, dim, dt, 3), table, lens, st)
    c.same()
    for i in range(4):
        lens = lens + 1
        c.write(*rows(6, heads, dim, dt, 10 + i), table, lens, kv.starts_of([1] * 6), null_start=True)
        c.same()


def test_token_by_token(w):
    """Every position of a page, its scale growing now and then."""
    rng = np.random.default_rng(0)
    c = Cache(w, 8, 2, 64, 32, 1)
    table = kv.make_table([100, 70], 32, 8, rng)
    for t in range(70):
        c.write(*rows(2, 2, 64, BF, t, spread=1.5), table, [t + 31, t + 1], kv.starts_of([1, 1]),
                null_start=True)
    c.same()


def test_again_is_the_same(w):
    """Writing the same rows again changes nothing, and after a step back the new rows replace."""
    rng = np.random.default_rng(0)
    c = Cache(w, 9, 2, 128, 16, 1)
    table = kv.make_table([40, 50], 16, 9, rng)
    st = kv.starts_of([21, 30])
    k, v = rows(51, 2, 128, F, 4)
    c.write(k, v, table, [40, 50], st)
    before = c.kv.clone(), c.sc.clone()
    w.kv8_write(k, v, c.kv, c.sc, dev(table), dev(np.array([40, 50], np.int32)), dev(st))
    assert torch.equal(before[0], c.kv) and torch.equal(before[1], c.sc)
    c.write(*rows(13, 2, 128, F, 5), table, [37, 45], kv.starts_of([6, 7]))
    c.same()


@pytest.mark.parametrize("dt", [BF, F])
def test_extremes(w, dt):
    """Zeros, values whose scale or inverse leaves the normal range, the largest ones."""
    c = Cache(w, 6, 1, 32, 16, 1)
    table = kv.make_table([96], 16, 6, np.random.default_rng(0))
    k, v = (x.contiguous() for x in rows(96, 1, 32, F, 6, spread=0.0))
    big = torch.finfo(dt).max
    for i, f in enumerate([0.0, 2.0 ** -149, 1e-40, 2e-38, 1e-36, 1.0]):
        k[16 * i:16 * i + 16] *= f
        v[16 * (5 - i):16 * (5 - i) + 16] *= f
    k[95, 0, 3] = big
    v[3, 0, 3] = -big
    c.write(k.to(dt), v.to(dt), table, [96], kv.starts_of([96]))
    c.same()
    # a zero page that grows, a tiny one that grows to the largest
    c.write(*(x[:1].to(dt) for x in (k, v)), table, [18], kv.starts_of([1]))
    c.same()


def test_pages_that_are_none(w):
    """Entries outside the cache, tables that end early, rows of no token: nothing is written."""
    c = Cache(w, 5, 2, 64, 16, 3)
    table = np.array([[0, -1, 2], [5, 2 ** 31 - 1, -2 ** 31], [3, 4, 1]], np.int32)
    k, v = rows(120, 2, 64, BF, 7)
    c.write(k, v, table, [48, 48, 80], kv.starts_of([48, 48, 24]))
    c.same()
    c.write(k[:9], v[:9], table, [0, -5, 4], kv.starts_of([2, 1, 6]))
    c.same()


def test_wide_tables_and_strides(w):
    c = Cache(w, 40, 2, 96, 16, 3)
    rng = np.random.default_rng(0)
    lens, n = [33, 100, 47], [33, 90, 1]
    whole = np.full((5, 11), 2 ** 30, np.int32)
    whole[1:4, 2:9] = kv.make_table(lens, 16, 40, rng, blocks=7)
    t = dev(whole)[1:4, 2:9]
    assert not t.is_contiguous() and t.data_ptr() % 16
    st = kv.starts_of(n)
    k, v = rows(124, 2, 96, BF, 8)
    w.kv8_write(k, v, c.kv, c.sc, t, dev(np.array(lens, np.int32)), dev(st))
    kv.write(c.codes, c.scales, whole[1:4, 2:9], lens, st, [x.float().cpu().numpy() for x in (k, v)])
    c.same()


@pytest.mark.parametrize("dim,page", [(32, 16), (64, 64), (96, 32), (128, 16), (128, 128), (256, 64)])
@pytest.mark.parametrize("dt", [BF, F])
def test_read(w, dim, page, dt):
    print("CASE kv8 read", dim, page, dt, flush=True)
    c = Cache(w, 40, 3, dim, page, 5)
    rng = np.random.default_rng(1)
    lens, n = [1, 150, 0, 77, 33], [1, 150, 2, 20, 0]
    table = kv.make_table(lens, page, 40, rng, blocks=-(-150 // page) + 1)
    table[3, 60 // page] = 40                                # no page: zeros
    st = kv.starts_of(n)
    total = int(st[-1])
    want = kv.read(c.codes, c.scales, table, lens, st, total + 3)
    k = torch.full((total + 3, 3, dim), float("nan"), dtype=dt, device="cuda")
    v = torch.full((total + 3, 4, dim), float("nan"), dtype=dt, device="cuda")[:, :3]
    gk, gv = w.kv8_read(c.kv, c.sc, dev(table), dev(np.array(lens, np.int32)), dev(st), k=k, v=v)
    assert gk is k
    for got, ref in ((gk, want[0]), (gv, want[1])):
        ref = torch.from_numpy(ref).to(dt)
        assert torch.equal(got.cpu().nan_to_num(9999), ref.nan_to_num(9999))
    if dt == BF:                                             # the last token of each
        lens = [5, 150, 70, 77, 33]
        a, b = w.kv8_read(c.kv, c.sc, dev(table), dev(np.array(lens, np.int32)))
        ref = kv.read(c.codes, c.scales, table, lens, kv.starts_of([1] * 5), 5)
        assert torch.equal(a.cpu(), torch.from_numpy(ref[0]).to(BF))
        assert torch.equal(b.cpu(), torch.from_numpy(ref[1]).to(BF))


def test_empty(w):
    c = Cache(w, 4, 2, 64, 16, 5)
    none = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    t0 = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    l0 = torch.empty((0,), dtype=torch.int32, device="cuda")
    w.kv8_write(none, none, c.kv, c.sc, t0, l0)
    assert w.kv8_read(c.kv, c.sc, t0, l0)[0].shape == (0, 2, 64)
    c.same()
    kv0, sc0 = w.kv8_cache(0, 2, 64, 16)                     # a cache without pages
    t, n = dev(np.zeros((2, 1), np.int32)), dev(np.array([3, 1], np.int32))
    k, v = rows(2, 2, 64, BF, 1)
    w.kv8_write(k, v, kv0, sc0, t, n)
    assert (w.kv8_read(kv0, sc0, t, n)[0] == 0).all()
    w.kv8_write(k, v, c.kv, c.sc, t[:, :0], n)               # tables without entries
    c.same()


def test_past_4_gib(w):
    """Pages whose bytes lie past 4 GiB (and past 2^32 elements)."""
    heads, dim, page = 8, 256, 128
    pages = (5 << 30) // (heads * 2 * page * dim) + 2
    kvt = torch.empty((pages, heads, 2, page, dim), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((pages, heads, 2), device="cuda")
    kvt[-3:] = 0
    table = dev(np.array([[pages - 1, pages - 3]], np.int32))
    k, v = rows(200, heads, dim, BF, 3)
    lens, st = dev(np.array([200], np.int32)), dev(np.array([0, 200], np.int32))
    w.kv8_write(k, v, kvt, sc, table, lens, st)
    small, ssc = w.kv8_cache(2, heads, dim, page)
    w.kv8_write(k, v, small, ssc, dev(np.array([[1, 0]], np.int32)), lens, st)
    assert torch.equal(kvt[pages - 1], small[1]) and torch.equal(kvt[pages - 3, :, :, :], small[0])
    a = w.kv8_read(kvt, sc, table, lens, st, tokens=200)
    b = w.kv8_read(small, ssc, dev(np.array([[1, 0]], np.int32)), lens, st, tokens=200)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals(w):
    c = Cache(w, 4, 2, 64, 16, 5)
    k, v = rows(3, 2, 64, BF, 1)
    t, n = dev(np.zeros((3, 2), np.int32)), dev(np.array([3, 1, 2], np.int32))
    good = dict(k=k, v=v, kv=c.kv, kv_scale=c.sc, block_table=t, lens=n, row_start=None)
    for bad in (dict(v=v[:2]), dict(v=v.float()), dict(k=k[:, :1]), dict(k=k[..., :32], v=v[..., :32]),
                dict(kv=c.kv.view(-1)), dict(kv=c.kv.view(torch.int8)), dict(kv_scale=c.sc[:3]),
                dict(block_table=t.long()), dict(block_table=t[:2]), dict(lens=n.long()),
                dict(lens=n[:2]), dict(row_start=n), dict(k=k[:2], v=v[:2]), dict(k=k.half(), v=v.half())):
        with pytest.raises((ValueError, w.W4A8Error)):
            w.kv8_write(**{**good, **bad})
    with pytest.raises(ValueError):
        w.kv8_read(c.kv, c.sc, t, n, dev(np.zeros(4, np.int32)))
    with pytest.raises(ValueError):
        w.kv8_read(c.kv, c.sc, t, n, out_dtype=torch.float16)
    c.same()


def test_graph(w):
    """Captured writes and reads follow what their arrays hold at each replay."""
    c = Cache(w, 30, 2, 128, 16, 5)
    table = kv.make_table([120, 90, 60], 16, 30, np.random.default_rng(2))
    k, v = (x.contiguous() for x in rows(3, 2, 128, BF, 0))
    lens, t = dev(np.array([100, 80, 50], np.int32)), dev(table)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.kv8_write(k, v, c.kv, c.sc, t, lens)
        w.kv8_read(c.kv, c.sc, t, lens, k=ko, v=vo)
    for i in range(5):
        nk, nv = rows(3, 2, 128, BF, 20 + i, spread=2.0)
        k.copy_(nk), v.copy_(nv)
        lens += 1
        graph.replay()
        host = lens.cpu().numpy()
        st = kv.starts_of([1] * 3)
        kv.write(c.codes, c.scales, table, host, st, [x.float().cpu().numpy() for x in (nk, nv)])
        c.same()
        want = kv.read(c.codes, c.scales, table, host, st, 3)
        assert torch.equal(ko.cpu(), torch.from_numpy(want[0]).to(BF))
        assert torch.equal(vo.cpu(), torch.from_numpy(want[1]).to(BF))

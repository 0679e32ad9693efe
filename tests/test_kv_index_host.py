"""The index arithmetic of the paged cache, compiled for the host: every page and row of a
ragged batch is visited exactly once, and whatever the arrays hold, no index leaves them."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import kv8_util as kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("kv") / "kv_index.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover", "-static-libubsan", "-I",
                    os.path.join(ROOT, "w4a8_quantized_gemm_quantize_amd", "csrc"),
                    os.path.join(ROOT, "tests", "kv_index_host.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.page_items.argtypes = [P, P, P, I64] + [I32] * 5 + [P]
    L.page_items.restype = I64
    L.tile_items.argtypes = [P, P, P, I64] + [I32] * 11 + [P]
    L.tile_items.restype = I64
    return L


def addr(a):
    return None if a is None else a.ctypes.data


def pages_of(lib, starts, lens, table, pages, rows, page):
    shift = page.bit_length() - 1
    args = [addr(starts), addr(lens), addr(table), table.shape[1], len(lens), table.shape[1], pages,
            rows, shift]
    out = np.zeros((lib.page_items(*args, None), 4), np.int64)
    lib.page_items(*args, addr(out))
    return out


def tiles_of(lib, starts, lens, table, pages, rows, page, tiles, group, shift, max_rows, causal=1,
             window=0):
    args = [addr(starts), addr(lens), addr(table), table.shape[1], len(lens), table.shape[1], pages,
            rows, page.bit_length() - 1, tiles, group, shift, max_rows, causal, window]
    out = np.zeros((lib.tile_items(*args, None), 8), np.int64)
    lib.tile_items(*args, addr(out))
    return out


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_layout(lib, dim):
    for t in range(0, 48, 5):
        for d in range(dim):
            if d % 8 == 0:
                assert lib.key_offset(t, d, dim) == kv.key_offset(t, d, dim)
            assert lib.value_offset(t, d, dim) == kv.value_offset(t, d, dim)
    for at in kv.offsets(32, dim):
        assert sorted(at.reshape(-1)) == list(range(32 * dim))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("seed", range(6))
def test_every_page_once(lib, page, seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 20))
    rows = rng.integers(0, [2, 5, 40, 200, 500, 3][seed], n)
    lens = (rows + rng.integers(0, 300, n) * (rng.random(n) < 0.7)).astype(np.int32)
    lens[rng.random(n) < 0.1] = 0                           # rows without a token
    table = kv.make_table(lens, page, int(sum(-(-x // page) for x in lens)) + 1, rng)
    starts = kv.starts_of(rows)
    got = pages_of(lib, starts, lens, table, 1 << 20, int(starts[-1]) + 3, page)
    want = []
    for s in range(n):
        lo = int(lens[s]) - int(rows[s])
        for b in range(max(lo, 0) // page, -(-int(lens[s]) // page) if rows[s] else 0):
            a, z = max(lo, b * page, 0), min(int(lens[s]), (b + 1) * page)
            if z > a:
                want.append((table[s, b], a - b * page, z - b * page, starts[s] + a - lo))
    assert sorted(map(tuple, got[got[:, 2] > got[:, 1]])) == sorted(want)


@pytest.mark.parametrize("seed", range(4))
def test_one_row_a_sequence(lib, seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 100, 30).astype(np.int32)
    table = kv.make_table(lens, 16, 400, rng)
    got = pages_of(lib, None, lens, table, 400, 30, 16)
    assert len(got) == 30
    for s, (p, first, last, row) in enumerate(got):
        if lens[s] == 0:
            assert last == first
        else:
            at = int(lens[s]) - 1
            assert (p, first, last, row) == (table[s, at // 16], at % 16, at % 16 + 1, s)


@pytest.mark.parametrize("group,shift", [(1, 4), (3, 4), (8, 4), (5, 6), (7, 7), (64, 4), (1, 8)])
@pytest.mark.parametrize("seed", range(4))
def test_every_row_in_one_tile(lib, group, shift, seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 12))
    rows = rng.integers(0, [2, 30, 300, 9][seed], n)
    lens = (rows + rng.integers(0, 50, n)).astype(np.int32)
    table = kv.make_table(lens, 16, 4000, rng)
    starts = kv.starts_of(rows)
    for max_rows in (int(max(rows.max(), 1)), 7):
        for tiles in (0, -(-min(max_rows, int(rows.max()) or 1) * group // (1 << shift))):
            got = tiles_of(lib, starts, lens, table, 4000, int(starts[-1]), 16, tiles, group, shift,
                           max_rows)
            seen = []
            for ok, s, first, m, row0, r, lo, hi in got:
                if not ok:
                    continue
                assert (first, m, lo) == (starts[s], rows[s], 0) and 0 < r <= 1 << shift
                assert hi == lens[s] - m + (row0 + r - 1) // group + 1
                seen += [(s, row0 + i) for i in range(r)]
            want = [(s, i) for s in range(n) for i in range(min(int(rows[s]), max_rows) * group)]
            assert sorted(seen) == want


def test_seen_tokens(lib):
    lens, table = np.array([100], np.int32), np.zeros((1, 5), np.int32)     # 80 tokens have places
    starts = np.array([0, 40], np.int32)
    def one(**kw):
        return [tuple(t[4:]) for t in tiles_of(lib, starts, lens, table, 1, 40, 16, 0, 2, 4, 40, **kw)
                if t[0]]
    assert one() == [(0, 16, 0, 68), (16, 16, 0, 76), (32, 16, 0, 80), (48, 16, 0, 80),
                     (64, 16, 0, 80)]
    assert [t[2:] for t in one(window=10)] == [(51, 68), (59, 76), (67, 80), (75, 80), (80, 80)]
    assert [t[2:] for t in one(causal=0)] == [(0, 80)] * 5
    starts, lens = np.array([0, 40], np.int32), np.array([10], np.int32)    # 30 rows of no token
    assert [t[2:] for t in one()][:4] == [(0, 0)] * 3 + [(0, 2)]


@pytest.mark.parametrize("seed", range(40))
def test_whatever_the_arrays_hold(lib, seed):
    """Row numbers stay in the batch, pages in the cache, tokens in the page."""
    rng = np.random.default_rng(seed)
    n, rows, page, pages = int(rng.integers(1, 9)), int(rng.integers(1, 300)), 32, 7
    wild = np.array([-2**31, -2**31 + 1, -1, 0, 1, 31, 32, 299, 2**31 - 1])

    def some(shape, hi):
        a = rng.integers(-3, hi, shape)
        return np.where(rng.random(shape) < 0.4, rng.choice(wild, shape), a).astype(np.int32)

    starts, lens, table = some(n + 1, rows + 5), some(n, 400), some((n, 6), pages + 3)
    got = pages_of(lib, starts, lens, table, pages, rows, page)
    live = got[got[:, 2] > got[:, 1]]
    assert (live[:, 0] >= -1).all() and (live[:, 0] < pages).all()
    assert (live[:, 1] >= 0).all() and (live[:, 2] <= page).all()
    assert (live[:, 3] >= 0).all() and (live[:, 3] + live[:, 2] - live[:, 1] <= rows).all()
    assert (got[got[:, 2] <= got[:, 1], 0] == -1).all()
    for group in (1, 5):
        for causal, window in ((1, 0), (0, 0), (1, 9), (0, 1 << 30)):
            t = tiles_of(lib, starts, lens, table, pages, rows, page, 0, group, 4, rows, causal, window)
            t = t[t[:, 0] > 0]
            last = t[:, 2] + (t[:, 4] + t[:, 5] - 1) // group
            assert (t[:, 2] >= 0).all() and (last < rows).all() and (t[:, 5] <= 16).all()
            assert (0 <= t[:, 6]).all() and (t[:, 6] <= t[:, 7]).all() and (t[:, 7] <= 6 * page).all()

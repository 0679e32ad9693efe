"""Debug mode of the attention set checks the rows that a call uses, and no others: a padded
batch whose tail was never written runs as it does without debug mode."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture()
def w(monkeypatch):
    from w4a8_quantized_gemm_quantize_amd import binding
    torch.cuda.init()
    monkeypatch.setenv("W4A8_DEBUG", "1")
    return binding


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def refused(w, call):
    with pytest.raises(w.W4A8Error) as e:
        call()
    assert e.value.status == w.ERR_NONFINITE


def some(rows, heads, dt, *bad):
    t = torch.ones((rows, heads, 64), dtype=dt, device="cuda")
    for r in bad:
        t[r, -1, 3] = NAN
    return t


@pytest.mark.parametrize("dt", [BF, F])
def test_rotation(w, dt):
    table = torch.zeros((10, 64), device="cuda")
    pos = ints(3, -1, 9, 10, 0)                              # rows 1 and 3 are left alone
    for bad in (1, 3):
        w.qk_norm_rope(some(5, 4, dt, bad), some(5, 2, dt, 1, 3), table, pos)
    for bad in (0, 2, 4):
        refused(w, lambda: w.qk_norm_rope(some(5, 4, dt, bad), some(5, 2, dt), table, pos))
        refused(w, lambda: w.qk_norm_rope(some(5, 4, dt), some(5, 2, dt, bad), table, pos))
    refused(w, lambda: w.qk_norm_rope(some(5, 4, dt, 1), some(5, 2, dt)))    # no rotation: all rows


# sequences of 3, 0, 4 and 20 rows: rows 0 .. 26 of 30.  The third has 2 tokens, so that its rows
# 3 and 4 have none; the fourth's second page is none: its tokens 16 .. 19, rows 23 .. 26.
START, LENS, TABLE = (0, 3, 3, 7, 27), (40, 5, 2, 20), ((0, 1, 2), (3, -1, -1), (4, -1, -1), (5, 9, -1))
UNUSED = {"write": (3, 4, 23, 26, 27, 29), "attn": (3, 4, 27, 29)}
USED = {"write": (0, 2, 5, 6, 7, 22), "attn": (0, 2, 5, 6, 7, 22, 26)}


def batch(w):
    kv, sc = w.kv8_cache(6, 2, 64, 16)
    return kv, sc, torch.tensor(TABLE, dtype=torch.int32, device="cuda"), ints(*LENS), ints(*START)


@pytest.mark.parametrize("dt", [BF, F])
def test_write(w, dt):
    kv, sc, table, lens, start = batch(w)
    w.kv8_write(some(30, 2, dt, *UNUSED["write"]), some(30, 2, dt, *UNUSED["write"]), kv, sc, table, lens,
                start)
    assert sc[[0, 1]].eq(0).all() and sc[[2, 4, 5]].gt(0).all()
    before = kv.clone(), sc.clone()
    for bad in USED["write"]:
        for k, v in ((some(30, 2, dt, bad), some(30, 2, dt)), (some(30, 2, dt), some(30, 2, dt, bad))):
            refused(w, lambda: w.kv8_write(k, v, kv, sc, table, lens, start))
    assert torch.equal(kv, before[0]) and torch.equal(sc, before[1])


@pytest.mark.parametrize("window", [0, 3])
def test_attention(w, window):
    kv, sc, table, lens, start = batch(w)
    unused, used = list(UNUSED["attn"]), list(USED["attn"])
    if window:                                               # tokens 18 and 19 see 16 .. 19 only
        unused += [25, 26]
        used.remove(26)
    out = w.attn_kv8(some(30, 4, BF, *unused), kv, sc, table, lens, start, window=window)
    assert torch.isfinite(out[:27]).all()
    for bad in used:
        refused(w, lambda: w.attn_kv8(some(30, 4, BF, bad), kv, sc, table, lens, start, window=window))
    # past max_rows
    w.attn_kv8(some(30, 4, BF, 2, 9, 26), kv, sc, table, lens, start, max_rows=2)
    refused(w, lambda: w.attn_kv8(some(30, 4, BF, 8), kv, sc, table, lens, start, max_rows=2))
    # without `causal` a row of no token sees what there is
    refused(w, lambda: w.attn_kv8(some(30, 4, BF, 3), kv, sc, table, lens, start, causal=False))


def test_single_tokens(w):
    kv, sc = w.kv8_cache(3, 2, 64, 16)
    wide = torch.full((3, 5), 7, dtype=torch.int32, device="cuda")
    table = wide[:, 1:3]
    table.copy_(torch.tensor([[0, 1], [-1, 2], [2, 0]]))
    lens = ints(17, 3, 0)                                    # the second's page is none, the third is empty
    w.kv8_write(some(3, 2, BF, 1, 2), some(3, 2, BF, 1, 2), kv, sc, table, lens)
    w.attn_kv8(some(3, 4, BF, 1, 2), kv, sc, table, lens)
    refused(w, lambda: w.kv8_write(some(3, 2, BF, 0), some(3, 2, BF), kv, sc, table, lens))
    refused(w, lambda: w.attn_kv8(some(3, 4, BF, 0), kv, sc, table, lens))

"""Attention over the 8-bit cache at the edges of what its entry point takes: caches without a
page in every form."""
import pytest

from test_gpu_attn_kv8 import Case, halves, w  # noqa: F401

pytestmark = pytest.mark.gpu


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

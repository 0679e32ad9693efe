"""Debug mode of the attention set: inputs that hold NaN or Inf are refused and nothing is
written; values between the rows of a strided tensor are not inputs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture()
def w(monkeypatch):
    from w4a8_quantized_gemm_quantize_amd import binding
    torch.cuda.init()
    monkeypatch.setenv("W4A8_DEBUG", "1")
    return binding


def setup(bad):
    rows = torch.ones((5, 8 * 64 + 8), dtype=BF, device="cuda")
    rows[:, 8 * 64:] = float("nan")                      # not part of any tensor below
    q, k, v = (rows[:, i * 64:j * 64].view(5, j - i, 64) for i, j in ((0, 4), (4, 6), (6, 8)))
    if bad is not None:
        {"q": q, "k": k, "v": v}[bad][3, 1, 5] = float("inf")
    table = torch.arange(5, dtype=torch.int32, device="cuda").view(5, 1)
    lens = torch.tensor([1, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    return q, k, v, table, lens


@pytest.mark.parametrize("bad", [None, "q", "k", "v"])
def test_refused(w, bad):
    q, k, v, table, lens = setup(bad)
    kv, sc = w.kv8_cache(5, 2, 64, 16)
    ang = torch.zeros((10, 64), device="cuda")
    calls = {
        "qk": lambda: w.qk_norm_rope(q, k, ang, lens, torch.ones(64, device="cuda")),
        "kv": lambda: w.kv8_write(k, v, kv, sc, table, lens),
        "q": lambda: w.attn_kv8(q, kv, sc, table, lens),
    }
    for reads, call in calls.items():
        if bad is not None and bad in reads:
            with pytest.raises(w.W4A8Error) as e:
                call()
            assert e.value.status == w.ERR_NONFINITE
            assert not kv.any() or reads != "kv"
        else:
            call()
    if bad == "q":
        weight = torch.full((64,), float("nan"), device="cuda")
        with pytest.raises(w.W4A8Error):
            w.qk_norm_rope(k, k.clone(), ang, lens, weight)

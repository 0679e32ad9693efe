"""Block tables wider than 32 bits are refused, not taken modulo 2^32."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("blocks", [(1 << 31) + 1, (1 << 32) + 2])
def test_wide_tables(blocks):
    from w4a8_quantized_gemm_quantize_amd import binding as w
    kv, sc = w.kv8_cache(2, 2, 32, 16)
    table = torch.empty((1, blocks), dtype=torch.int32, device="cuda")
    table[0, :2] = torch.arange(2, dtype=torch.int32, device="cuda")
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    k = torch.ones((1, 2, 32), dtype=BF, device="cuda")
    for call in (lambda t: w.kv8_write(k, k, kv, sc, t, lens), lambda t: w.kv8_read(kv, sc, t, lens),
                 lambda t: w.attn_kv8(k, kv, sc, t, lens)):
        with pytest.raises(w.W4A8Error) as e:
            call(table)
        assert e.value.status == w.ERR_UNSUPPORTED
    assert not kv.any()
    w.kv8_write(k, k, kv, sc, table[:, :2], lens)            # two entries of it are a table
    assert kv.any()

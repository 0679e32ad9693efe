"""w4a8_moe_ffn refuses sizes whose products would need more work items than a launch holds
(2^32: 2^22 tiles of 256 x 256 in workgroups of 1024), before anything is launched.  The
pointers are fake and never dereferenced."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "w4a8_quantized_gemm_quantize_amd", "libw4a8.so")
UNSUPPORTED, BF16, A = 3, 1, 0x10000

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libw4a8.so not built")


@pytest.fixture(scope="module")
def lib():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding._lib


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter,fits", [
    ((1 << 25) - 1, 8, 32, 64, 64, False),          # 2^22 + 7 row tiles, one column tile
    ((1 << 25) - 4096, 8, 32, 64, 64, True),
    ((1 << 23) - 1, 1, 32, 128, 512, False),        # 2^20 row tiles, four column tiles
    ((1 << 23) - 4096, 1, 32, 128, 512, True),
    ((1 << 23) - 1, 1, 32, 128, 384, True),
])
def test_work_items(lib, tokens, experts, top_k, hidden, inter, fits):
    need = lib.w4a8_moe_ffn_workspace_bytes(tokens, experts, top_k, hidden, inter, BF16)
    assert (need > 0) == fits
    if not fits:
        assert lib.w4a8_moe_ffn(*[A] * 9, tokens, experts, top_k, hidden, inter, 64, A, BF16, A,
                                1 << 62, None) == UNSUPPORTED

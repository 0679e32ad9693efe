"""The workspace tells in how many parts the tokens of a batch are taken: the sizes that the GPU
tests of long sequences run are split, in each of the forms that they stand for."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "w4a8_quantized_gemm_quantize_amd", "libw4a8.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libw4a8.so not built")


@pytest.mark.parametrize("rows,height", [(1, 16), (3, 16), (16, 32), (100, 128)])
def test_long_sequences_are_split(rows, height):
    """Two sequences of `rows` rows over 30000 tokens, 8 query heads over 2 of 128."""
    from w4a8_quantized_gemm_quantize_amd import binding as w
    need = w.attn_kv8_workspace_bytes(2 * rows, 2, True, rows, -(-(30011 + rows) // 64), 8, 2, 128, 64)
    tiles = min(2 * -(-rows * 4 // height), 2 * rows * 4 // height + 2)
    parts, rest = divmod(need, tiles * 2 * height * (128 + 4) * 4)
    assert rest == 0 and parts > 8                          # joined a wavefront a row

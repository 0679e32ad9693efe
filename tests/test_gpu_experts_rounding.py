"""w4a8_moe_ffn rounds its output once: the bf16 output is the binary32 layer, put together
from w4a8_gemm expert by expert, rounded to the nearest bf16, bit for bit, whichever form
the sizes choose."""
import pytest
import torch

from test_gpu_experts import CASES, composed, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding


# sizes that choose the tiled kernels at few rows (64-wide rows) and at many
ROUNDING = CASES + [(1, 1, 1, 64, 64), (5, 3, 2, 64, 192), (4, 3, 2, 192, 64), (90, 4, 3, 128, 128)]


@pytest.mark.parametrize("case", ROUNDING, ids=lambda c: "-".join(map(str, c)))
def test_bf16_output_is_rounded_once(w, case):
    print(case, flush=True)
    x, ids, wts, w13, w2 = make(w, *case, seed=sum(case) + 1)
    wts = wts - 0.5                                  # slots that cancel
    got = w.w4a8_moe_ffn(x, ids, wts, w13, w2, case[4])
    want = composed(w, x, ids, wts, w13, w2, case[4])
    assert torch.equal(got, want.to(torch.bfloat16))


def test_a_token_keeps_its_bits_in_a_larger_batch(w):
    """64-row tiles and the skinny kernels give a token the same bf16 bits."""
    x, ids, wts, w13, w2 = make(w, 300, 4, 2, 256, 192, seed=3)
    large = w.w4a8_moe_ffn(x, ids, wts, w13, w2, 192)
    for t in (1, 12, 40):
        few = w.w4a8_moe_ffn(x[:t], ids[:t], wts[:t], w13, w2, 192)
        assert torch.equal(few, large[:t]), t

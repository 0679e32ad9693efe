"""lora_add keeps all 24 bits of a x up to the sum with y, for both output types.

Every value, product and partial sum below is a multiple of 2^-20 of magnitude below 2, so
it is exact in binary32 in any order: the result is exact, and what is left after y cancels
the leading bits is the last bits of a x."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t", [1, 20, 64, 65, 200])
@pytest.mark.parametrize("rank,k", [(8, 64), (24, 64), (64, 256), (128, 64), (8, 40960)])
def test_last_bits_of_the_first_product_arrive(w, dtype, t, rank, k):
    n = 72
    x = torch.ones((t, k), dtype=torch.bfloat16)
    a = torch.zeros((2, rank, k))
    a[:, 0, :3] = torch.tensor([1.0, 2.0 ** -9, 2.0 ** -20])      # v0 = 1 + 2^-9 + 2^-20
    a[:, rank - 1, k - 1] = 1.0                                     # v_last = 1
    b = torch.zeros((2, n, rank))
    b[:, :, 0] = 1.0
    b[:, :, rank - 1] = -2.0 ** -9
    y = torch.full((t, n), -1.0, dtype=dtype)
    ids = (torch.arange(t) % 2).to(torch.int32)
    out = w.lora_add(x.cuda(), a.to(torch.bfloat16).cuda(), b.to(torch.bfloat16).cuda(),
                     ids.cuda(), y.cuda())
    assert torch.equal(out.cpu(), torch.full((t, n), 2.0 ** -20, dtype=dtype))

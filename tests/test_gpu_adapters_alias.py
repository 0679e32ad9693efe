"""lora_add where out shares memory with x: every row is what separate tensors give.

Batches of few rows take one launch where the tensors are separate, whose workgroups read
all of x while others write out; shared ones may not.  Compared with 64 bits on copies of
the inputs, within test_gpu_adapters' bound."""
import pytest
import torch

from test_gpu_adapters import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding


SIZES = [(1, 2, 16, 4096), (8, 8, 16, 4096), (33, 5, 8, 2048), (64, 3, 32, 1024), (200, 4, 24, 1032)]


@pytest.mark.parametrize("t,adapters,rank,k", SIZES)
def test_one_tensor_for_x_y_and_out(w, t, adapters, rank, k):
    print(t, adapters, rank, k, flush=True)
    x, a, b, ids, _, s = make(t, adapters, rank, k, k, torch.bfloat16, seed=t + k)
    buf = x.cuda()
    got = w.lora_add(buf, a.cuda(), b.cuda(), ids.cuda(), buf, scale=s.cuda(), out=buf)
    assert got is buf
    check(buf, x, a, b, ids, x, s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 512, 1016])
@pytest.mark.parametrize("t", [3, 40, 100])
def test_out_over_part_of_x(w, dtype, shift, t):
    print(dtype, shift, t, flush=True)
    k, n = 1024, 1024
    x, a, b, ids, y, s = make(t, 3, 16, k, n, dtype, seed=shift + t)
    es = 2 if dtype == torch.bfloat16 else 4
    raw = torch.zeros((t, 3 * 4096), dtype=torch.uint8, device="cuda")
    xs = raw.view(torch.bfloat16)[:, :k]
    out = raw.view(dtype)[:, shift * 2 // es:shift * 2 // es + n]
    xs.copy_(x)
    got = w.lora_add(xs, a.cuda(), b.cuda(), ids.cuda(), y.cuda(), scale=s.cuda(), out=out)
    check(got, x, a, b, ids, y, s)


@pytest.mark.parametrize("t", [4, 100])
def test_interleaved_columns_share_nothing(w, t):
    x, a, b, ids, y, s = make(t, 3, 16, 512, 264, torch.bfloat16, seed=t)
    raw = torch.zeros((t, 512 + 264 + 264), dtype=torch.bfloat16, device="cuda")
    raw[:, 264:776], raw[:, 776:] = x.cuda(), y.cuda()
    args = a.cuda(), b.cuda(), ids.cuda()
    got = w.lora_add(raw[:, 264:776], *args, raw[:, 776:], scale=s.cuda(), out=raw[:, :264])
    assert torch.equal(got, w.lora_add(x.cuda(), *args, y.cuda(), scale=s.cuda()))
    assert torch.equal(raw[:, 264:776].cpu(), x) and torch.equal(raw[:, 776:].cpu(), y)

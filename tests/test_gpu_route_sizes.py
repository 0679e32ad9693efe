"""moe_route at the numbers of tokens that its limit (fewer than 2^31) admits: more than one
launch holds.  The keys are the logits, so the choice is exact; with top_k 1 a renormalized
weight is the scale."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding


@pytest.mark.parametrize("tokens", [(1 << 25) + 1, (1 << 26) + 7, (1 << 27) + 3])
def test_more_tokens_than_a_launch_holds(w, tokens):
    print(tokens, flush=True)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn((tokens, 2), generator=g, device="cuda", dtype=torch.float32)
    x = x.to(torch.bfloat16)
    ids = torch.full((tokens, 1), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((tokens, 1), -7.0, device="cuda")
    w.moe_route(x, 1, ids=ids, weights=weights, scale=1.5)
    want = (x[:, 1] > x[:, 0]).to(torch.int32)           # ties to the lower expert
    assert torch.equal(ids[:, 0], want)
    assert bool((weights == 1.5).all())

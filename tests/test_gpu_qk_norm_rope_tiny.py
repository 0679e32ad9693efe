"""Norms of rows whose mean square is subnormal, without an eps that hides it."""
import pytest
import torch

from test_gpu_qk_norm_rope import inputs, model, w  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dim", [8, 96, 128, 256])
@pytest.mark.parametrize("dt,size", [(F, 2.0 ** -62), (F, 2.0 ** -66), (BF, 2.0 ** -66), (F, 2.0 ** -70)])
def test_tiny_rows(w, dim, dt, size):
    """Squares and their mean round to multiples of 2^-149: each by 2^-150 at most, so the mean by
    2 * 2^-150, and its root by 2^-150 / mean relative to it, beside the bound of normal rows."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = [((1 + torch.rand((5, 3, dim), generator=g, device="cuda")) * size).to(dt) for _ in range(2)]
    _, _, wq, wk, _ = inputs(5, 3, 3, dim, F, 1)
    out = w.qk_norm_rope(x[0], x[1], q_weight=wq, k_weight=wk, eps=0.0, out_dtype=F)
    for got, x, weight in zip(out, x, (wq, wk)):
        y, err = model(x, weight, None, None, 0.0, False)
        err = err + y.abs() * 2.0 ** -150 / x.double().square().mean(-1, keepdim=True)
        off = (got.double() - y).abs()
        assert (off <= err * (1 + 2.0 ** -6) + 2.0 ** -24 * y.abs()).all(), (off / err).max().item()

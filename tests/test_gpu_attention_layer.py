"""The example layer (projection, norms and rotation, cache, attention, projection) runs
eagerly and captured, and is what its operators' formulas give one after the other."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv8_util as kv
from test_gpu_attn_kv8 import near
from test_gpu_qk_norm_rope import check, model

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_runs(example):
    out, worst = example.main(tokens=130, steps=5)
    assert out.shape == (130, 1024) and out.isfinite().all()
    assert worst == 0.0                              # replays give the eager bits


def test_layer_is_its_operators(example):
    """Prompts, a second chunk and decode steps through views of one projection's rows: each
    operator's outputs against its formula on what the one before it left, and the cache
    against its binary32 model all along."""
    from w4a8_quantized_gemm_quantize_amd import binding as w
    m = example.AttentionLayer(hidden=256, q_heads=6, kv_heads=2, head_dim=96, page=16, pages=40)
    reqs = example.Requests(3, 40, 16, 12)
    hq, hk, d = 6, 2, 96
    codes = np.zeros((2, 40, hk, 16, d), np.int8)
    codes[:] = kv.unpack(m.kv.cpu().numpy())
    scales = m.kv_scale.cpu().numpy().copy()
    g = torch.Generator(device="cuda").manual_seed(1)
    for counts in ([50, 7, 0], [20, 1, 33], [1, 1, 1], [1, 1, 1], [3, 0, 2]):
        past = list(reqs.host)
        start, pos = example.prompt_rows(counts, past)
        reqs.grow(counts)
        n = sum(counts)
        x = torch.randn((n, 256), generator=g, device="cuda").to(torch.bfloat16)
        qkv = w.w4a8_gemm_bf16act(x, *m.qkv, m.rows)
        raw = qkv.clone()
        q, k = qkv[:, :hq * d].view(n, hq, d), qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
        v = qkv[:, (hq + hk) * d:].view(n, hk, d)
        w.qk_norm_rope(q, k, m.cos_sin, pos, m.q_norm, m.k_norm, q_out=q, k_out=k)
        check(q, *model(raw[:, :hq * d].view(n, hq, d), m.q_norm, m.cos_sin, pos, 1e-6, False), "q")
        check(k, *model(raw[:, hq * d:(hq + hk) * d].view(n, hk, d), m.k_norm, m.cos_sin, pos, 1e-6,
                        False), "k")
        assert torch.equal(v.reshape(n, -1), raw[:, (hq + hk) * d:])
        # the layer itself does the writing
        out = m(x, pos, reqs.table, reqs.lens, start, max_rows=max(counts))
        table, lens = reqs.table.cpu().numpy(), list(reqs.host)
        st = start.cpu().numpy()
        kv.write(codes, scales, table, lens, st, [t.float().cpu().numpy() for t in (k, v)])
        assert np.array_equal(kv.unpack(m.kv.cpu().numpy()), codes)
        assert np.array_equal(m.kv_scale.cpu().numpy(), scales)
        att, lse = w.attn_kv8(q, m.kv, m.kv_scale, reqs.table, reqs.lens, start,
                              max_rows=max(counts), want_lse=True)
        near(att, lse, *kv.attention(q, torch.from_numpy(codes).cuda(),
                                     torch.from_numpy(scales).cuda(), table, lens, st))
        assert torch.equal(out, w.w4a8_gemm_bf16act(att.view(n, hq * d), *m.proj, 256))
        # what was written reads back
        rk, rv = w.kv8_read(m.kv, m.kv_scale, reqs.table, reqs.lens, start, tokens=n,
                            out_dtype=torch.float32)
        want = kv.read(codes, scales, table, lens, st, n)
        assert np.array_equal(rk.cpu().numpy(), want[0]) and np.array_equal(rv.cpu().numpy(), want[1])

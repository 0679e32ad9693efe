"""Host-side checks of the row-selected entry points: invalid arguments are refused with
the documented status before anything is launched, and empty batches do nothing.  The
pointers are fake and never dereferenced."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "w4a8_quantized_gemm_quantize_amd", "libw4a8.so")
OK, NULL, SHAPE, UNSUPPORTED, MISALIGNED = range(5)
A, MIS = 0x10000, 0x10008
F32, BF16, I32 = range(3)

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libw4a8.so not built")


@pytest.fixture(scope="module")
def lib():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding._lib


def route(lib, **kw):
    a = dict(logits=A, dtype=F32, ld=64, bias=A, tokens=4, experts=64, top_k=8, score=0, groups=8,
             topk_groups=4, group_top=2, renorm=1, scale=1.0, ids=A, weights=A, stream=None)
    a.update(kw)
    return lib.w4a8_moe_route(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK),
    (dict(tokens=0, logits=None, ids=None, weights=None), OK),
    (dict(tokens=-1), SHAPE),
    (dict(experts=0), SHAPE),
    (dict(top_k=0), SHAPE),
    (dict(ld=63), SHAPE),
    (dict(groups=0), SHAPE),
    (dict(groups=7), SHAPE),
    (dict(topk_groups=0), SHAPE),
    (dict(topk_groups=9), SHAPE),
    (dict(topk_groups=1, top_k=9), SHAPE),          # a group has 8
    (dict(group_top=0), UNSUPPORTED),
    (dict(group_top=3), UNSUPPORTED),
    (dict(experts=1032, ld=1032), UNSUPPORTED),
    (dict(top_k=33, topk_groups=8), UNSUPPORTED),
    (dict(experts=65, ld=65, groups=65, topk_groups=65), UNSUPPORTED),
    (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(dtype=I32), UNSUPPORTED),
    (dict(score=2), UNSUPPORTED),
    (dict(logits=None), NULL),
    (dict(ids=None), NULL),
    (dict(weights=None), NULL),
    (dict(logits=MIS), MISALIGNED),
    (dict(bias=MIS), MISALIGNED),
    (dict(ids=MIS), MISALIGNED),
    (dict(weights=MIS), MISALIGNED),
])
def test_route_refusals(lib, kw, want):
    assert route(lib, **kw) == want


def moe(lib, **kw):
    a = dict(x=A, ids=A, weights=A, p13=A, g13=A, c13=A, p2=A, g2=A, c2=A, tokens=4, experts=8,
             top_k=2, hidden=256, inter=128, group=64, out=A, dtype=BF16, ws=A, ws_bytes=1 << 40,
             stream=None)
    a.update(kw)
    return lib.w4a8_moe_ffn(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK),
    (dict(tokens=0, x=None, out=None, ws=None, ws_bytes=0), OK),
    (dict(tokens=-1), SHAPE),
    (dict(experts=0), SHAPE),
    (dict(top_k=0), SHAPE),
    (dict(hidden=0), SHAPE),
    (dict(inter=0), SHAPE),
    (dict(hidden=96), SHAPE),
    (dict(inter=96), SHAPE),
    (dict(group=32), UNSUPPORTED),
    (dict(dtype=I32), UNSUPPORTED),
    (dict(experts=1025), UNSUPPORTED),
    (dict(top_k=33), UNSUPPORTED),
    (dict(hidden=150976 + 64), UNSUPPORTED),
    (dict(inter=150976 + 64), UNSUPPORTED),
    (dict(hidden=65536, inter=65536), UNSUPPORTED),     # 2^32 weights in one matrix
    (dict(tokens=(1 << 31) // 256), UNSUPPORTED),       # x has 2^31 elements
    (dict(tokens=1 << 27, top_k=32, hidden=64), UNSUPPORTED),
    (dict(ws_bytes=1024), SHAPE),
    (dict(ws=MIS), MISALIGNED),
] + [({n: None}, NULL) for n in ("x", "ids", "weights", "p13", "g13", "c13", "p2", "g2", "c2",
                                 "out", "ws")]
  + [({n: MIS}, MISALIGNED) for n in ("x", "ids", "weights", "p13", "g13", "c13", "p2", "g2",
                                      "c2", "out")])
def test_moe_refusals(lib, kw, want):
    assert moe(lib, **kw) == want


def test_moe_workspace(lib):
    need = lib.w4a8_moe_ffn_workspace_bytes(4, 8, 2, 256, 128, BF16)
    assert need >= 8 * 128 * 2                         # h of every slot
    assert moe(lib, ws_bytes=need - 1) == SHAPE
    assert lib.w4a8_moe_ffn_workspace_bytes(0, 8, 2, 256, 128, BF16) == 0
    assert lib.w4a8_moe_ffn_workspace_bytes(4, 8, 2, 250, 128, BF16) == 0
    assert lib.w4a8_moe_ffn_workspace_bytes(4, 8, 2, 256, 128, F32) >= need


def lora(lib, **kw):
    a = dict(x=A, ldx=256, a=A, b=A, scale=A, ids=A, tokens=4, adapters=3, rank=16, k=256, n=128,
             y=A, ldy=128, out=0x90000, ldo=128, dtype=BF16, ws=A, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.w4a8_lora_add(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK),
    (dict(tokens=0, x=None, y=None, ws=None), OK),
    (dict(tokens=-1), SHAPE),
    (dict(adapters=0), SHAPE),
    (dict(rank=0), SHAPE),
    (dict(rank=12), SHAPE),
    (dict(k=252), SHAPE),
    (dict(n=124), SHAPE),
    (dict(n=0), SHAPE),
    (dict(ldx=248), SHAPE),
    (dict(ldx=260), SHAPE),
    (dict(ldy=120), SHAPE),
    (dict(ldo=132), SHAPE),
    (dict(out=A, ldo=136), SHAPE),                      # in place with another stride
    (dict(rank=136), UNSUPPORTED),
    (dict(adapters=4096), UNSUPPORTED),
    (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(n=1 << 24, ldy=1 << 24, ldo=1 << 24), UNSUPPORTED),
    (dict(k=(1 << 30) + 8, ldx=1 << 31), UNSUPPORTED),
    (dict(dtype=I32), UNSUPPORTED),
    (dict(ws_bytes=64), SHAPE),
    (dict(scale=MIS), MISALIGNED),
] + [({n: None}, NULL) for n in ("x", "a", "b", "ids", "y", "out", "ws")]
  + [({n: MIS}, MISALIGNED) for n in ("x", "a", "b", "ids", "y", "out", "ws")])
def test_lora_refusals(lib, kw, want):
    assert lora(lib, **kw) == want


def test_lora_workspace(lib):
    for tokens in (1, 64, 65, 5000):
        need = lib.w4a8_lora_workspace_bytes(tokens, 3, 16, 256)
        assert need > 0
        assert lora(lib, tokens=tokens, ws_bytes=need - 1) == SHAPE
    assert lib.w4a8_lora_workspace_bytes(4, 3, 12, 256) == 0


def test_binding_refuses_wrong_tensors():
    import torch
    from w4a8_quantized_gemm_quantize_amd import binding
    host = torch.zeros((2, 8))
    with pytest.raises(ValueError):
        binding.moe_route(host, 2)                     # not on the GPU
    with pytest.raises(ValueError):
        binding.moe_route(host, 2, score="tanh")
    with pytest.raises(ValueError):
        binding.w4a8_moe_ffn(host, host, host, (host,) * 3, (host,) * 3, 64)
    with pytest.raises(ValueError):
        binding.lora_add(host, host, host, host, host)

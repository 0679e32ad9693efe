"""Host-side checks of the cache's and attention's entry points: invalid arguments are refused
with the documented status before anything is launched, and empty batches do nothing.  The
pointers are fake and never dereferenced."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "w4a8_quantized_gemm_quantize_amd", "libw4a8.so")
OK, NULL, SHAPE, UNSUPPORTED, MISALIGNED = range(5)
A, MIS, ODD = 0x10000, 0x10008, 0x10002
F32, BF16, I32 = range(3)

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libw4a8.so not built")


@pytest.fixture(scope="module")
def lib():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding._lib


def rope(lib, **kw):
    a = dict(q=A, ldq=6144, k=A, ldk=6144, in_dtype=BF16, qw=A, kw=A, eps=1e-6, table=A, pos=A,
             max_pos=100, rot=128, interleaved=0, tokens=3, q_heads=32, kv_heads=8, dim=128, qo=0x90000,
             ldqo=4096, ko=0xa0000, ldko=1024, out_dtype=BF16, stream=None)
    a.update(kw)
    return lib.w4a8_qk_norm_rope(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK),
    (dict(tokens=0, q=None, k=None, qo=None, ko=None, table=None, pos=None), OK),
    (dict(tokens=-1), SHAPE),
    (dict(q_heads=-1), SHAPE),
    (dict(q_heads=0, kv_heads=0), SHAPE),
    (dict(dim=0), SHAPE),
    (dict(dim=100), SHAPE),
    (dict(rot=-8), SHAPE),
    (dict(rot=136), SHAPE),
    (dict(rot=12), SHAPE),
    (dict(max_pos=-1), SHAPE),
    (dict(ldq=4088), SHAPE),
    (dict(ldk=1028), SHAPE),
    (dict(ldqo=4095), SHAPE),
    (dict(ldko=1020), SHAPE),
    (dict(out_dtype=F32, ldqo=4098), SHAPE),
    (dict(qo=A), SHAPE),                               # in place with another stride
    (dict(qo=A, ldqo=6144, out_dtype=F32), SHAPE),     # in place with another type
    (dict(ko=A), SHAPE),
    (dict(dim=264, ldq=1 << 16, ldk=1 << 16, ldqo=1 << 16, ldko=1 << 16), UNSUPPORTED),
    (dict(in_dtype=I32), UNSUPPORTED),
    (dict(out_dtype=I32), UNSUPPORTED),
    (dict(tokens=1 << 24), UNSUPPORTED),
    (dict(tokens=1 << 23, q_heads=64, ldq=16384, ldqo=8192), UNSUPPORTED),
    (dict(q=MIS), MISALIGNED), (dict(k=MIS), MISALIGNED), (dict(qo=MIS), MISALIGNED),
    (dict(ko=MIS), MISALIGNED), (dict(qw=MIS), MISALIGNED), (dict(kw=MIS), MISALIGNED),
    (dict(table=MIS), MISALIGNED), (dict(pos=ODD), MISALIGNED),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(qo=None), NULL), (dict(ko=None), NULL),
    (dict(pos=None), NULL), (dict(table=None), NULL),
])
def test_rope_refusals(lib, kw, want):
    assert rope(lib, **kw) == want


BATCH = dict(table=A, ldb=10, blocks=8, lens=A, start=A, seqs=2, rows=5)
CACHE = dict(kv_heads=4, dim=128, page=16, pages=100)

# what the three calls on the cache refuse alike
COMMON = [
    (dict(rows=0), OK),
    (dict(seqs=0), OK),
    (dict(rows=-1), SHAPE),
    (dict(seqs=-1), SHAPE),
    (dict(blocks=-1), SHAPE),
    (dict(ldb=7), SHAPE),
    (dict(kv_heads=0), SHAPE),
    (dict(dim=0), SHAPE),
    (dict(dim=48), SHAPE),
    (dict(page=0), SHAPE),
    (dict(pages=-1), SHAPE),
    (dict(start=None), SHAPE),                         # rows are not one a sequence
    (dict(dim=288), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED),
    (dict(page=48), UNSUPPORTED),
    (dict(page=256), UNSUPPORTED),
    (dict(kv_heads=1025), UNSUPPORTED),
    (dict(pages=1 << 31), UNSUPPORTED),
    (dict(blocks=(1 << 26) + 1, ldb=1 << 27), UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(seqs=(1 << 30) + 1), UNSUPPORTED),
    (dict(lens=None), NULL),
    (dict(table=None), NULL),
    (dict(kv=None), NULL),
    (dict(kv_scale=None), NULL),
    (dict(lens=ODD), MISALIGNED),
    (dict(table=ODD), MISALIGNED),
    (dict(start=ODD), MISALIGNED),
    (dict(kv=MIS), MISALIGNED),
    (dict(kv_scale=MIS), MISALIGNED),
]


def write(lib, **kw):
    a = dict(k=A, ldk=512, v=A, ldv=520, dtype=BF16, **BATCH, **CACHE, kv=A, kv_scale=A, stream=None)
    a.update(kw)
    return lib.w4a8_kv8_write(*a.values())


def read(lib, **kw):
    a = dict(kv=A, kv_scale=A, **BATCH, **CACHE, k=A, ldk=512, v=A, ldv=520, dtype=BF16, stream=None)
    a.update(kw)
    return lib.w4a8_kv8_read(*a.values())


ROWS = COMMON + [
    (dict(dtype=I32), UNSUPPORTED),
    (dict(ldk=504), SHAPE),
    (dict(ldv=516), SHAPE),
    (dict(dtype=F32, ldv=518), SHAPE),
    (dict(rows=1 << 28, kv_heads=16, ldk=2048, ldv=2048), UNSUPPORTED),     # workgroups
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=MIS), MISALIGNED), (dict(v=MIS), MISALIGNED),
]


@pytest.mark.parametrize("kw,want", ROWS)
def test_write_refusals(lib, kw, want):
    assert write(lib, **kw) == want


@pytest.mark.parametrize("kw,want", ROWS)
def test_read_refusals(lib, kw, want):
    assert read(lib, **kw) == want


def attn(lib, **kw):
    a = dict(q=A, ldq=1536, kv=A, kv_scale=A, table=A, ldb=10, blocks=8, lens=A, start=A, seqs=2,
             rows=5, max_rows=4, q_heads=12, kv_heads=4, dim=128, page=16, pages=100, causal=1,
             window=0, scale=0.1, out=0x90000, ldo=1536, lse=A, ws=A, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.w4a8_attn_kv8(*a.values())


@pytest.mark.parametrize("kw,want", [(k, w) for k, w in COMMON if k.get("kv_heads") not in (0, 1025)] + [
    (dict(kv_heads=0), SHAPE),
    (dict(kv_heads=1025, q_heads=1025), UNSUPPORTED),
    (dict(q_heads=0), SHAPE),
    (dict(q_heads=13), SHAPE),
    (dict(q_heads=4 * 65, ldq=1 << 16, ldo=1 << 16), UNSUPPORTED),
    (dict(rows=1 << 29, q_heads=64, ldq=1 << 16, ldo=1 << 16), UNSUPPORTED),
    (dict(rows=1 << 28, max_rows=1 << 28), UNSUPPORTED),                    # workgroups
    (dict(max_rows=0), SHAPE),
    (dict(window=-1), SHAPE),
    (dict(window=(1 << 30) + 1), UNSUPPORTED),
    (dict(ldq=1528), SHAPE),
    (dict(ldo=1540), SHAPE),
    (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(q=MIS), MISALIGNED), (dict(out=MIS), MISALIGNED), (dict(lse=MIS), MISALIGNED),
])
def test_attn_refusals(lib, kw, want):
    assert attn(lib, **kw) == want


def test_attn_workspace(lib):
    def need(rows, seqs, ragged, max_rows, blocks, q_heads=32, kv_heads=8, dim=128, page=16):
        return lib.w4a8_attn_kv8_workspace_bytes(rows, seqs, ragged, max_rows, blocks, q_heads,
                                                 kv_heads, dim, page)
    assert need(1, 1, 0, 1, 4) == 0                        # 64 tokens are not split
    w = need(1, 1, 0, 1, 4096)
    assert w > 0
    big = dict(blocks=4096, ldb=4096, seqs=1, rows=1, max_rows=1, start=None, q_heads=32, kv_heads=8,
               ldq=4096, ldo=4096)
    assert attn(lib, **big, ws_bytes=w - 1) == SHAPE
    assert attn(lib, **big, ws=None) == NULL
    assert attn(lib, **big, ws=MIS) == MISALIGNED
    assert need(0, 1, 1, 1, 4096) == 0 and need(1, 0, 1, 1, 4096) == 0
    assert need(5, 2, 1, 0, 4096) == 0 and need(1, 1, 0, 1, 4096, dim=100) == 0
    assert need(2, 1, 0, 1, 4096) == 0                     # not one row a sequence


def test_binding_refuses_wrong_tensors():
    import torch
    from w4a8_quantized_gemm_quantize_amd import binding as b
    host = torch.zeros((2, 4, 64))
    kv, sc = b.kv8_cache(3, 4, 64, 16, device="cpu")
    assert kv.shape == (3, 4, 2, 16, 64) and kv.dtype == torch.uint8 and sc.shape == (3, 4, 2)
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        b.qk_norm_rope(host, host)
    with pytest.raises(ValueError):
        b.kv8_write(host, host, kv, sc, table, lens)
    with pytest.raises(ValueError):
        b.kv8_read(kv, sc, table, lens)
    with pytest.raises(ValueError):
        b.attn_kv8(host.to(torch.bfloat16), kv, sc, table, lens)

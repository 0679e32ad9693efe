"""lora_add against a plain implementation in 64 bits.

Tolerance per element, with S = |scale| |b| (|a| |x|) (the sum of the magnitudes of all
terms): a x is summed in binary32 in chains of at most k / 128 + 40 additions, the
expand sum in at most rank / 8 + 10, each within 2^-24 of the running magnitude; v is
split to 2^-16 (bf16 outputs) or 2^-24; the output is rounded once (2^-8 or 2^-24).  The
matrix cores' internal sums of 32 products are taken as 4 more roundings per step."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding


def make(t, adapters, rank, k, n, dtype, seed, ids=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((t, k), generator=g).to(torch.bfloat16)
    a = (torch.randn((adapters, rank, k), generator=g) * k ** -0.5).to(torch.bfloat16)
    b = torch.randn((adapters, n, rank), generator=g).to(torch.bfloat16)
    y = torch.randn((t, n), generator=g).to(dtype)
    s = torch.rand((adapters,), generator=g) * 3 - 1
    if ids is None:
        ids = torch.randint(-1, adapters + 1, (t,), generator=g)     # both ends: no adapter
    return x, a, b, ids.to(torch.int32), y, s


def reference(x, a, b, ids, y, s):
    x, a, b, y = (v.double() for v in (x, a, b, y))
    s = torch.ones(len(a)) if s is None else s
    out, mag = y.clone(), torch.zeros_like(y)
    for l in range(len(a)):
        r = (ids == l).nonzero()[:, 0]
        out[r] += float(s[l]) * ((x[r] @ a[l].T) @ b[l].T)
        mag[r] += abs(float(s[l])) * ((x[r].abs() @ a[l].abs().T) @ b[l].abs().T)
    return out, mag


def check(got, x, a, b, ids, y, s):
    want, mag = reference(x, a, b, ids, y, s)
    k, rank = x.shape[1], a.shape[1]
    bf = y.dtype == torch.bfloat16
    rel = (4 * (k / 128 + 40) + rank / 8 + 10) * 2.0 ** -24 + 2.0 ** (-16 if bf else -24)
    tol = rel * mag + want.abs() * 2.0 ** (-8 if bf else -24) * 1.01 + 1e-30
    err = (got.cpu().double() - want).abs()
    assert (err <= tol).all(), f"{float((err / tol).max()):.3f} of the bound"
    none = (ids < 0) | (ids >= len(a))
    assert torch.equal(got.cpu()[none], y[none]), "rows without an adapter keep y"


CASES = [
    # tokens, adapters, rank, k, n
    (1, 1, 8, 8, 8),
    (1, 4, 16, 4096, 4096),
    (2, 3, 24, 200, 72),
    (16, 1, 16, 512, 264),
    (17, 2, 32, 1000, 520),
    (63, 40, 64, 2048, 1032),
    (60, 7, 16, 4000, 1504),
    (64, 5, 16, 1024, 10000),
    (40, 9, 32, 5000, 1000),        # two launches for decode batches, by what they read
    (60, 7, 16, 9600, 1504),
    (64, 5, 8, 9600, 8200),         # several column steps in a workgroup
    (64, 2, 128, 776, 248),
    (65, 2, 128, 776, 248),
    (65, 70, 8, 136, 1000),
    (130, 1, 40, 4104, 56),
    (300, 5, 16, 9000, 600),
    (1025, 33, 72, 640, 328),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_lora_matches_64_bits(w, case, dtype):
    print(case, dtype, flush=True)
    v = make(*case, dtype, seed=sum(case))
    x, a, b, ids, y, s = (t.cuda() for t in v)
    got = w.lora_add(x, a, b, ids, y, scale=s)
    check(got, *v)
    assert torch.equal(got, w.lora_add(x, a, b, ids, y, scale=s)), "same call, same bits"
    check(w.lora_add(x, a, b, ids, y), *v[:5], None)


@pytest.mark.parametrize("t", [40, 200])
@pytest.mark.parametrize("fill", [-1, 0, 2], ids=["no adapter", "first", "last"])
def test_batches_of_one_kind(w, t, fill):
    v = make(t, 3, 16, 264, 136, torch.float32, 5, ids=torch.full((t,), fill))
    x, a, b, ids, y, s = (q.cuda() for q in v)
    check(w.lora_add(x, a, b, ids, y, scale=s), *v)


@pytest.mark.parametrize("t", [33, 150])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_strides_in_place_and_streams(w, t, dtype):
    v = make(t, 4, 32, 320, 200, dtype, 9)
    x, a, b, ids, y, s = (q.cuda() for q in v)
    want = w.lora_add(x, a, b, ids, y, scale=s)
    wide_x = torch.full((t, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_x[:, 64:384] = x
    wide_y = torch.full((t, 600), float("nan"), dtype=dtype, device="cuda")
    wide_y[:, 200:400] = y
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w.lora_add(wide_x[:, 64:384], a, b, ids, wide_y[:, 200:400], scale=s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    view = wide_y[:, 200:400]
    assert w.lora_add(x, a, b, ids, view, scale=s, out=view) is view        # in place
    assert torch.equal(view, want)
    assert wide_y[:, :200].isnan().all() and wide_y[:, 400:].isnan().all()


@pytest.mark.parametrize("t", [20, 100])
def test_values_that_are_not_numbers_stay_in_their_rows(w, t):
    x, a, b, ids, y, s = make(t, 3, 24, 136, 72, torch.float32, 11)
    ids[:] = torch.arange(t) % 3
    x[5] = float("nan")
    x[7, 3] = float("inf")
    a[2] = float("nan")                              # an adapter that is broken
    got = w.lora_add(x.cuda(), a.cuda(), b.cuda(), ids.cuda(), y.cuda(), scale=s.cuda()).cpu()
    good = torch.ones(t, dtype=torch.bool)
    good[[5, 7]] = False
    good &= ids != 2
    clean = a.clone()
    clean[2] = 0
    check(got[good], x[good], clean, b, ids[good], y[good], s)
    assert got[5].isnan().all()


@pytest.mark.parametrize("t", [3, 70])
def test_adapters_past_4_gib(w, t):
    a = torch.zeros((610, 128, 28672), dtype=torch.bfloat16, device="cuda")      # 4.5 GB
    b = torch.zeros((610, 64, 128), dtype=torch.bfloat16, device="cuda")
    x, a1, b1, ids, y, s = make(t, 1, 128, 28672, 64, torch.float32, 3, ids=torch.zeros(t))
    a[609], b[609] = a1[0].cuda(), b1[0].cuda()
    got = w.lora_add(x.cuda(), a, b, torch.full((t,), 609, dtype=torch.int32, device="cuda"),
                     y.cuda())
    check(got, x, a1, b1, ids, y, None)


def test_refusals_on_the_device(w):
    v = make(4, 2, 16, 64, 32, torch.bfloat16, 1)
    x, a, b, ids, y, s = (q.cuda() for q in v)
    with pytest.raises(w.W4A8SizeError):
        w.lora_add(x, a, b, ids[:3], y)
    with pytest.raises(w.W4A8SizeError):
        w.lora_add(x, a, b, ids, y[:3])
    with pytest.raises(w.W4A8SizeError):
        w.lora_add(x, a, b, ids, y, scale=s[:1])
    with pytest.raises(ValueError):
        w.lora_add(x, a, b[:1], ids, y)
    with pytest.raises(ValueError):
        w.lora_add(x, a, b, ids, y.half())
    with pytest.raises(w.W4A8Error) as err:
        w.lora_add(x[:, 1:57], a[:, :, :56].contiguous(), b, ids, y)      # misaligned rows
    assert err.value.status == w.ERR_MISALIGNED
    with pytest.raises(w.W4A8Error) as err:
        w.lora_add(x, a[:, :12].contiguous(), b[:, :, :12].contiguous(), ids, y)
    assert err.value.status == w.ERR_SHAPE
    with pytest.raises(w.W4A8Error) as err:
        w.lora_add(x, a, b, ids, y,
                   workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert err.value.status == w.ERR_SHAPE
    assert w.lora_add(x[:0], a, b, ids[:0], y[:0]).shape == (0, 32)

"""w4a8_moe_ffn against a plain implementation in 64 bits, and bit for bit against the
same layer put together from w4a8_gemm, expert by expert.

The 64-bit form takes the codes of x from binary32 products, as defined; its h differs
from the kernel's binary32 steps by at most about 8 ulp, so now and then an h rounds to
the neighbouring bf16 value and its code moves by one.  Tight bound of an element: y
carries at most 8 roundings of binary32 and, for bf16 outputs, one of bf16 each, the
output one more.  A slot with a moved code adds at most 112 hs c |w| per code; at most a
tenth of the slots move, by at most three codes together."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding


def make(w, t, e, k, hidden, inter, seed, unused=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((t, hidden), generator=g, device="cuda").to(torch.bfloat16)
    popular = torch.rand((e,), generator=g, device="cuda") ** 3 + 1e-3
    ids = torch.multinomial(popular.expand(t, e), k, replacement=k > e, generator=g)
    ids[torch.rand(ids.shape, generator=g, device="cuda") < unused] = -1
    ids[torch.rand(ids.shape, generator=g, device="cuda") < unused / 4] = e
    wts = torch.rand((t, k), generator=g, device="cuda")

    def weights(n, kk):
        m = (0.02 * torch.randn((e * n, kk), generator=g, device="cuda")).to(torch.bfloat16)
        return w.pack_w4_grouped(m)

    return x, ids.to(torch.int32), wts, weights(2 * inter, hidden), weights(hidden, inter)


def int_weights(w, packed, n, k):
    q, s = w.unpack_w4_grouped(packed[0], packed[1], n, k)
    return (q.double().view(n, -1, 64) * s.double()[..., None]).view(n, k).cpu().numpy()


def codes(v):
    """v float32 [rows, n] -> codes and scales (both float64), binary32 steps."""
    amax = np.abs(v).max(1, keepdims=True).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.where(amax > 0, np.float32(127) * (np.float32(1) / amax), np.float32(0))
    q = np.rint((v * inv.astype(np.float32)).astype(np.float32))
    s = amax * np.float32(np.float32(1) / np.float32(127))
    return q.astype(np.float64), s.astype(np.float64)


def bf16(v):
    return torch.from_numpy(v).to(torch.bfloat16).float().numpy()


def check64(w, x, ids, wts, w13, w2, inter, out):
    t, hidden = x.shape
    e = w13[2].numel() // (2 * inter)
    i13 = int_weights(w, w13, e * 2 * inter, hidden).reshape(e, 2 * inter, hidden)
    i2 = int_weights(w, w2, e * hidden, inter).reshape(e, hidden, inter)
    c13 = w13[2].cpu().double().numpy().reshape(e, -1)
    c2 = w2[2].cpu().double().numpy().reshape(e, -1)
    q, s = codes(x.float().cpu().numpy())
    idn, wn = ids.cpu().numpy(), wts.cpu().double().numpy()
    want = np.zeros((t, hidden))
    mag, move = np.zeros((t, hidden)), np.zeros((t, hidden))
    for ex in range(e):
        tok, slot = np.nonzero(idn == ex)
        if not len(tok):
            continue
        gu = (q[tok] @ i13[ex].T) * s[tok] * c13[ex]
        g, u = gu[:, :inter], gu[:, inter:]
        h = bf16(g / (1 + np.exp(-g)) * u)
        hq, hs = codes(h)
        y = (hq @ i2[ex].T) * hs * c2[ex] * wn[tok, slot][:, None]
        np.add.at(want, tok, y)
        np.add.at(mag, tok, np.abs(y))
        np.add.at(move, tok, 112 * 3 * hs * c2[ex] * np.abs(wn[tok, slot])[:, None])
    bf = out.dtype == torch.bfloat16
    got = out.double().cpu().numpy()
    err = np.abs(got - want)
    tight = mag * (2.0 ** -20 + (2.0 ** -8 if bf else 0)) + np.abs(want) * (
        2.0 ** -8 * 1.01 if bf else 0) + 1e-30
    assert (err <= tight + move).all()
    loose = (err > tight).any(1)
    assert loose.sum() <= max(1, 0.1 * (idn >= 0).sum()), (loose.sum(), t)
    assert (got[((idn < 0) | (idn >= e)).all(1)] == 0).all(), "tokens without experts"


def composed(w, x, ids, wts, w13, w2, inter):
    """The layer from the library's own products, binary32 output."""
    t, hidden = x.shape
    k = ids.shape[1]
    e = w13[2].numel() // (2 * inter)

    def part(packed, ex, n, kk):
        p, g, c = packed
        return (p[ex * n * kk // 2:(ex + 1) * n * kk // 2].clone(),
                g[ex * n * kk // 64:(ex + 1) * n * kk // 64].clone(), c[ex * n:(ex + 1) * n].clone())

    def quant(v):
        v = v.float()
        amax = v.abs().amax(1, keepdim=True)
        inv = torch.where(amax > 0, torch.full_like(amax, 127.0) * (torch.ones_like(amax) / amax),
                          torch.zeros_like(amax))
        q = torch.round(v * inv).nan_to_num(0.0).to(torch.int8)
        return q, (amax * torch.tensor(1 / 127, device=v.device))[:, 0].contiguous()

    q, s = quant(x)
    y = torch.zeros((t, k, hidden), device="cuda")
    for ex in range(e):
        tok, slot = (ids == ex).nonzero(as_tuple=True)
        if not len(tok):
            continue
        gu = w.w4a8_gemm(q[tok].contiguous(), s[tok].contiguous(), *part(w13, ex, 2 * inter, hidden),
                         2 * inter, out_dtype=torch.float32)
        g, u = gu[:, :inter], gu[:, inter:]
        h = (g / (torch.ones_like(g) + torch.exp(-g)) * u).to(torch.bfloat16)
        hq, hs = quant(h)
        y[tok, slot] = w.w4a8_gemm(hq, hs, *part(w2, ex, hidden, inter), hidden,
                                   out_dtype=torch.float32)
    out = torch.zeros((t, hidden), device="cuda")
    for j in range(k):
        used = ((ids[:, j] >= 0) & (ids[:, j] < e))[:, None]
        out = torch.where(used, out + wts[:, j, None] * y[:, j], out)
    return out


CASES = [
    # tokens, experts, top_k, hidden, inter
    (1, 1, 1, 64, 64),
    (1, 16, 4, 256, 192),
    (3, 5, 5, 192, 64),
    (8, 64, 8, 512, 128),
    (40, 6, 3, 320, 448),
    (33, 200, 2, 128, 320),
    (1, 9, 3, 1088, 192),           # few rows: taken one by one
    (2, 64, 8, 320, 4160),
    (3, 128, 20, 128, 2112),
    (1, 8, 8, 128, 14336),
    (1, 32, 32, 64 + 64, 16384),
    (30, 8, 1, 512, 2112),          # fused down product, then with codes from memory
    (60, 8, 2, 4160, 1088),
    (20, 10, 2, 192, 8256),
    (150, 4, 2, 448, 256),          # about 64 rows an expert
    (301, 7, 4, 256, 320),          # 128-row tiles
    (700, 2, 2, 320, 192),          # 256-row tiles
    (17, 3, 7, 128, 128),           # the same expert twice in a token
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_layer(w, case):
    print(case, flush=True)
    x, ids, wts, w13, w2 = make(w, *case, seed=sum(case))
    inter = case[4]
    out = w.w4a8_moe_ffn(x, ids, wts, w13, w2, inter, out_dtype=torch.float32)
    assert torch.equal(out, composed(w, x, ids, wts, w13, w2, inter))
    check64(w, x, ids, wts, w13, w2, inter, out)
    half = w.w4a8_moe_ffn(x, ids, wts, w13, w2, inter)
    assert half.dtype == torch.bfloat16
    check64(w, x, ids, wts, w13, w2, inter, half)


@pytest.mark.parametrize("t", [1, 5, 90, 700])
def test_one_expert_takes_all_and_others_none(w, t):
    x, ids, wts, w13, w2 = make(w, t, 4, 2, 192, 128, seed=t, unused=0)
    for fill in (0, 3):
        ids.fill_(fill)
        out = w.w4a8_moe_ffn(x, ids, wts, w13, w2, 128, out_dtype=torch.float32)
        assert torch.equal(out, composed(w, x, ids, wts, w13, w2, 128))
    ids.fill_(-1)
    out = torch.full((t, 192), float("nan"), device="cuda")
    w.w4a8_moe_ffn(x, ids, wts, w13, w2, 128, out=out)
    assert (out == 0).all()


def test_rows_of_zeros_and_large_values(w):
    x, ids, wts, w13, w2 = make(w, 20, 3, 2, 256, 128, seed=1)
    x[3] = 0
    x[5] *= 1e4
    x[6] *= 1e-4
    out = w.w4a8_moe_ffn(x, ids, wts, w13, w2, 128, out_dtype=torch.float32)
    assert torch.equal(out, composed(w, x, ids, wts, w13, w2, 128))
    assert (out[3] == 0).all() and out.isfinite().all()


@pytest.mark.parametrize("t", [4, 120])
def test_workspace_reuse_streams_and_repeats(w, t):
    x, ids, wts, w13, w2 = make(w, t, 8, 2, 320, 192, seed=7)
    want = w.w4a8_moe_ffn(x, ids, wts, w13, w2, 192, out_dtype=torch.float32)
    ws = torch.full((w.moe_ffn_workspace_bytes(t, 8, 2, 320, 192, torch.float32),), 0xff,
                    dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = w.w4a8_moe_ffn(x, ids, wts, w13, w2, 192, out_dtype=torch.float32, workspace=ws,
                             stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        ids2 = ids.flip(0).contiguous()
        other = w.w4a8_moe_ffn(x, ids2, wts, w13, w2, 192, out_dtype=torch.float32,
                               workspace=ws, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other, composed(w, x, ids2, wts, w13, w2, 192))


def test_captured_in_a_graph(w):
    x, ids, wts, w13, w2 = make(w, 6, 8, 2, 320, 192, seed=8)
    logits = torch.randn((6, 8), device="cuda")
    rid, rw = w.moe_route(logits, 2)
    out = torch.empty((6, 320), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(w.moe_ffn_workspace_bytes(6, 8, 2, 320, 192), dtype=torch.uint8,
                     device="cuda")

    def step():
        w.moe_route(logits, 2, ids=rid, weights=rw)
        w.w4a8_moe_ffn(x, rid, rw, w13, w2, 192, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        logits.copy_(torch.randn((6, 8), device="cuda"))
        x.copy_(torch.randn((6, 320), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out), i


def test_weights_past_4_gib(w):
    hidden, inter, e = 4096, 14336, 76               # 4.5 GB of gate and up weights
    g = torch.Generator(device="cuda").manual_seed(4)

    def stack(n, k):
        def nibbles():
            return torch.randint(1, 16, (e * n * k // 2,), generator=g, device="cuda",
                                 dtype=torch.uint8)
        packed = nibbles()
        packed |= nibbles() << 4
        s = torch.randint(1, 17, (e * n * k // 64,), generator=g, device="cuda",
                          dtype=torch.uint8)
        return packed, s, torch.full((e * n,), 5e-4, device="cuda")

    def pick(st, n, k, which):
        return tuple(torch.cat([t.view(e, -1)[i] for i in which]) for t in st)

    w13, w2 = stack(2 * inter, hidden), stack(hidden, inter)
    two13, two2 = (pick(st, n, k, (1, e - 1)) for st, n, k in ((w13, 2 * inter, hidden),
                                                              (w2, hidden, inter)))
    for t in (1, 12, 80, 900):
        x = torch.randn((t, hidden), generator=g, device="cuda").to(torch.bfloat16)
        few = torch.randint(0, 2, (t, 1), generator=g, device="cuda", dtype=torch.int32)
        wts = torch.rand((t, 1), generator=g, device="cuda")
        got = w.w4a8_moe_ffn(x, torch.where(few == 0, 1, e - 1).to(torch.int32), wts, w13, w2,
                             inter, out_dtype=torch.float32)
        # y is binary32 in both (the two forms of bf16 outputs may round y or not)
        assert torch.equal(got, w.w4a8_moe_ffn(x, few, wts, two13, two2, inter,
                                               out_dtype=torch.float32)), t


def test_refusals_on_the_device(w):
    x, ids, wts, w13, w2 = make(w, 4, 3, 2, 128, 64, seed=2)
    with pytest.raises(ValueError):
        w.w4a8_moe_ffn(x, ids[:3], wts, w13, w2, 64)
    with pytest.raises(w.W4A8SizeError):
        w.w4a8_moe_ffn(x, ids, wts[:3].contiguous(), w13, w2, 64)
    with pytest.raises(w.W4A8SizeError):
        w.w4a8_moe_ffn(x, ids, wts, w13, w2, 128)        # not a multiple of the stacked rows
    with pytest.raises(w.W4A8SizeError):
        w.w4a8_moe_ffn(x, ids, wts, w13, (w2[0][:-16], w2[1], w2[2]), 64)
    with pytest.raises(w.W4A8Error) as err:
        w.w4a8_moe_ffn(x, ids, wts, w13, w2, 64, workspace=torch.empty(
            64, dtype=torch.uint8, device="cuda"))
    assert err.value.status == w.ERR_SHAPE
    with pytest.raises(ValueError):
        w.w4a8_moe_ffn(x, ids.long(), wts, w13, w2, 64)
    assert w.w4a8_moe_ffn(x[:0], ids[:0], wts[:0], w13, w2, 64).shape == (0, 128)

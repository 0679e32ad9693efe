"""Every form of w4a8_moe_ffn (row by row; skinny with the down product's codes taken in the
product or from memory; 64- and 256-row tiles): on weights past 4 GiB, captured, with a
workspace used again, with long rows; and against 64 bits with a bound per element.

The form a case runs is told by its workspace, whose rule is restated here."""
import numpy as np
import pytest
import torch

from test_gpu_experts import codes, composed, int_weights, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    from w4a8_quantized_gemm_quantize_amd import binding
    return binding


def workspace(form, t, e, k, hidden, inter):
    """Bytes of a form: h always; else codes and scales of x, order and source of the sorted
    rows, the tile table, codes and scales of h (unless taken in the product), y."""
    rows = t * k
    bm = dict(few=16, few_fused=16, tile64=64, tile256=256).get(form)
    parts = [rows * inter * 2]
    if form != "direct":
        slots = rows // bm + min(rows, e)
        parts += [t * hidden, t * 4, rows * 4, rows * 4, (slots + 1) * 16, rows * hidden * 4]
        if form != "few_fused":
            parts += [rows * inter, rows * 4]
    return sum((p + 255) // 256 * 256 for p in parts)


def runs(w, form, t, e, k, hidden, inter):
    assert w.moe_ffn_workspace_bytes(t, e, k, hidden, inter) == workspace(form, t, e, k, hidden,
                                                                          inter), form


FORMS = [
    # form, tokens, experts, top_k, hidden, inter
    ("direct", 2, 16, 2, 512, 256),
    ("few_fused", 30, 6, 3, 512, 192),
    ("few", 24, 4, 2, 256, 4224),
    ("tile64", 100, 5, 3, 320, 192),
    ("tile64", 3, 4, 2, 64, 192),
    ("tile256", 400, 3, 2, 320, 192),
]


@pytest.mark.parametrize("case", FORMS, ids=lambda c: "-".join(map(str, c)))
def test_captured_and_workspace_used_again(w, case):
    form, t, e, k, hidden, inter = case
    print(case, flush=True)
    runs(w, *case)
    x, ids, wts, w13, w2 = make(w, t, e, k, hidden, inter, seed=t)
    ws = torch.full((w.moe_ffn_workspace_bytes(t, e, k, hidden, inter, torch.float32),), 0xff,
                    dtype=torch.uint8, device="cuda")
    out = torch.empty((t, hidden), device="cuda")

    def step():
        w.w4a8_moe_ffn(x, ids, wts, w13, w2, inter, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    assert torch.equal(out, composed(w, x, ids, wts, w13, w2, inter))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(t)
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        ids.copy_(torch.randint(-1, e + 1, ids.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        ws.fill_(0xff)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out), i
        assert torch.equal(got, composed(w, x, ids, wts, w13, w2, inter)), i


@pytest.mark.parametrize("case", [
    ("tile256", 900, 4, 2, 4160, 2112),         # 33 chunks of K, the last one half
    ("tile64", 500, 12, 2, 4160, 2112),
    ("few", 40, 4, 2, 7168, 4096),
    ("few_fused", 60, 256, 8, 7168, 256),
    ("tile64", 600, 256, 8, 7168, 256),
    ("direct", 1, 256, 8, 7168, 256),
], ids=lambda c: "-".join(map(str, c)))
def test_long_rows_and_many_experts(w, case):
    print(case, flush=True)
    runs(w, *case)
    x, ids, wts, w13, w2 = make(w, *case[1:], seed=7)
    out = w.w4a8_moe_ffn(x, ids, wts, w13, w2, case[5], out_dtype=torch.float32)
    assert torch.equal(out, composed(w, x, ids, wts, w13, w2, case[5]))


def test_both_stacks_past_4_gib(w):
    hidden, inter, e = 4096, 14336, 150          # 8.8 GB of gate and up weights, 4.4 of down
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

    def pick(st, which):
        return tuple(torch.cat([t.view(e, -1)[i] for i in which]) for t in st)

    w13, w2 = stack(2 * inter, hidden), stack(hidden, inter)
    two13, two2 = pick(w13, (1, e - 1)), pick(w2, (1, e - 1))
    for form, t in (("direct", 1), ("few", 40), ("tile64", 17 * e), ("tile256", 201 * e)):
        print(form, t, flush=True)
        runs(w, form, t, e, 1, hidden, inter)
        x = torch.randn((t, hidden), generator=g, device="cuda").to(torch.bfloat16)
        few = torch.randint(0, 2, (t, 1), generator=g, device="cuda", dtype=torch.int32)
        few[0] = 1
        wts = torch.rand((t, 1), generator=g, device="cuda")
        got = w.w4a8_moe_ffn(x, torch.where(few == 0, 1, e - 1).to(torch.int32), wts, w13, w2,
                             inter, out_dtype=torch.float32)
        assert torch.equal(got, w.w4a8_moe_ffn(x, few, wts, two13, two2, inter,
                                               out_dtype=torch.float32)), form


CASES64 = [
    # tokens, experts, top_k, hidden, inter
    (1, 9, 3, 1088, 192),
    (3, 128, 20, 128, 256),
    (1, 32, 32, 128, 512),
    (17, 3, 7, 128, 128),
    (30, 8, 1, 512, 576),
    (60, 8, 2, 1088, 320),
    (150, 4, 2, 448, 256),
    (700, 2, 2, 320, 192),
]


@pytest.mark.parametrize("case", CASES64, ids=lambda c: "-".join(map(str, c)))
def test_each_element_against_64_bits(w, case):
    """Bound of an element, u = 2^-24.  y takes three roundings (the sum to binary32, two
    scales), the weight one and the slots' sum one each: (top_k + 6) u of the magnitudes.
    An element of h is within (16 + 4 |g|) u of its 64-bit value (three roundings of each
    product, |g| times those through the exponential, exp 2 ulp, three more steps); where
    both ends of that window round to one bf16 value, so does the kernel's h.  Where they
    do not, its code may move by one (one bf16 step is less than one code), which moves
    column n by |W2[n, i]| hs c2; if the row's maximum itself is not sure, or more than
    that, the slot's whole scale may move: its magnitude times 2^-7 is added."""
    t, e, k, hidden, inter = case
    print(case, flush=True)
    u = 2.0 ** -24
    x, ids, wts, w13, w2 = make(w, *case, seed=sum(case) + 5)
    out = w.w4a8_moe_ffn(x, ids, wts, w13, w2, inter, out_dtype=torch.float32)
    i13 = int_weights(w, w13, e * 2 * inter, hidden).reshape(e, 2 * inter, hidden)
    i2 = int_weights(w, w2, e * hidden, inter).reshape(e, hidden, inter)
    c13 = w13[2].cpu().double().numpy().reshape(e, -1)
    c2 = w2[2].cpu().double().numpy().reshape(e, -1)
    q, s = codes(x.float().cpu().numpy())
    idn, wn = ids.cpu().numpy(), wts.cpu().double().numpy()

    def bf(v):
        return torch.from_numpy(v).to(torch.bfloat16).float().numpy()

    want, tol = np.zeros((t, hidden)), np.full((t, hidden), 1e-30)
    loose = 0
    for ex in range(e):
        tok, slot = np.nonzero(idn == ex)
        if not len(tok):
            continue
        gu = (q[tok] @ i13[ex].T) * s[tok] * c13[ex]
        gate, up = gu[:, :inter], gu[:, inter:]
        h64 = gate / (1 + np.exp(-gate)) * up
        win = (16 + 4 * np.abs(gate)) * u
        h = bf(h64)
        unsure = bf(h64 * (1 - win)) != bf(h64 * (1 + win))
        hq, hs = codes(h)
        scale = hs * c2[ex] * np.abs(wn[tok, slot])[:, None]
        y = (hq @ i2[ex].T) * hs * c2[ex] * wn[tok, slot][:, None]
        top = np.abs(h).max(1, keepdims=True)
        # the maximum moves only if an element that may move is within a step of it
        moved = (unsure & (np.abs(h) >= top * (1 - 2.0 ** -7))).any(1, keepdims=True)
        loose += int(moved.sum())
        mag = (np.abs(hq) @ np.abs(i2[ex]).T) * scale
        np.add.at(want, tok, y)
        np.add.at(tol, tok, np.abs(y) * (k + 6) * u + (unsure @ np.abs(i2[ex]).T) * scale
                  + moved * (mag * 2.0 ** -7 + np.abs(i2[ex]).sum(1) * scale))
    assert loose <= 0.1 * (idn >= 0).sum() + 1
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())


def test_codes_are_the_quantizers_but_at_halves(w):
    """The layer takes codes as rne(x * (127 * (1 / amax))), quantize_act_blockwise as
    rne(x * (127 / amax)) (test_layer holds the layer to the former bit for bit).  The two
    differ by one code, only where x * 127 / amax is exactly a half, and by one ulp of the
    scale."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn((512, 1024), generator=g).to(torch.bfloat16)
    q, s = codes(x.float().numpy())
    lib_q, lib_s = w.quantize_act_blockwise(x.cuda(), 1024)
    lib_q, lib_s = lib_q.cpu().numpy().astype(np.float64), lib_s.cpu().numpy()
    x64 = np.abs(x.double().numpy())
    amax = x64.max(1, keepdims=True)
    half = (np.fmod(x64 * 254, amax) == 0) & (np.fmod(np.round(x64 * 254 / amax), 2) == 1)
    differ = q != lib_q
    assert differ.any() and (half[differ]).all()
    assert np.abs(q - lib_q).max() == 1
    assert (np.abs(s - lib_s) <= np.spacing(np.maximum(s, lib_s).astype(np.float32))).all()

"""Norms of queries and keys with the rotation against the formula in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def w():
    from w4a8_quantized_gemm_quantize_amd import binding
    torch.cuda.init()
    return binding


def table(max_pos, rot, theta=1e4):
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * \
        theta ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / max(rot // 2, 1))
    return torch.cat([a.cos(), a.sin()], 1).float()


def model(x, weight, cs, pos, eps, interleaved):
    """(y, what its steps in binary32 may be off by), u = 2^-24 a rounding:
    the sum of head_dim squares and its root: (head_dim + 4) u / 2 + 2 u relative (a square
    root halves the relative error), two products more; then two products and a sum."""
    u = 2.0 ** -24
    y = x.double()
    rel = 0.0
    if weight is not None:
        r = 1 / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
        y = y * r * weight.double()
        rel = ((x.shape[-1] + 4) / 2 + 6) * u
    err = y.abs() * rel
    if cs is not None:
        rot = cs.shape[1]
        c = cs[pos.long()].double()[:, None]
        c, s = c[..., :rot // 2], c[..., rot // 2:]
        i = torch.arange(rot // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ya, yb, big = y[..., a], y[..., b], y.abs() * (rel + 3 * u)
        ea, eb = big[..., a], big[..., b]
        y, err = y.clone(), err.clone()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        err[..., a], err[..., b] = (ea * c.abs() + eb * s.abs()), (eb * c.abs() + ea * s.abs())
    return y, err


def check(got, y, err, name):
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny
    off = (got.double() - y).abs()
    room = err * (1 + half) + half * y.abs() + tiny
    assert (off <= room).all(), f"{name}: {(off / room).max().item()} of what it may be"


def inputs(tokens, hq, hk, dim, dt, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = (hq + 2 * hk) * dim + pad
    rows = torch.randn((tokens, n), generator=g, device="cuda") * \
        torch.exp(2 * torch.randn((tokens, 1), generator=g, device="cuda"))
    rows = rows.to(dt)
    q = rows[:, :hq * dim].view(tokens, hq, dim) if tokens else rows.new_empty((0, hq, dim))
    k = rows[:, hq * dim:(hq + hk) * dim].view(tokens, hk, dim) if tokens else rows.new_empty((0, hk, dim))
    wq, wk = (1 + 0.3 * torch.randn((dim,), generator=g, device="cuda") for _ in range(2))
    pos = torch.randint(0, 500, (tokens,), generator=g, device="cuda").to(torch.int32)
    return q, k, wq, wk, pos


CASES = [(1, 32, 8, 128, 128, False, BF, BF), (7, 14, 2, 96, 32, True, F, BF),
         (33, 5, 5, 64, 64, False, BF, F), (2, 1, 1, 8, 8, False, F, F), (3, 3, 1, 8, 8, True, BF, BF),
         (5, 9, 3, 256, 256, True, BF, BF), (5, 9, 3, 256, 64, False, F, F),
         (4, 17, 1, 192, 192, False, BF, BF), (4, 2, 2, 80, 40, False, BF, BF),
         (4, 33, 4, 72, 16, True, F, BF), (300, 64, 8, 128, 128, False, BF, BF),
         (601, 37, 3, 64, 64, False, BF, BF), (500, 13, 6, 256, 64, True, F, BF),
         (1, 1, 8, 128, 8, False, BF, BF)]


@pytest.mark.parametrize("tokens,hq,hk,dim,rot,inter,din,dout", CASES)
@pytest.mark.parametrize("norm", ["both", "none", "q"])
def test_formula(w, tokens, hq, hk, dim, rot, inter, din, dout, norm):
    print("CASE rope", tokens, hq, hk, dim, rot, inter, din, dout, norm, flush=True)
    q, k, wq, wk, pos = inputs(tokens, hq, hk, dim, din, dim + tokens)
    wq, wk = (wq if norm != "none" else None), (wk if norm == "both" else None)
    cs = table(500, rot)
    gq, gk = w.qk_norm_rope(q, k, cs, pos, wq, wk, eps=1e-5, interleaved=inter, out_dtype=dout)
    assert gq.dtype == dout and gq.shape == q.shape and gk.shape == k.shape
    check(gq, *model(q, wq, cs, pos, 1e-5, inter), "q")
    check(gk, *model(k, wk, cs, pos, 1e-5, inter), "k")


def test_norm_alone(w):
    q, k, wq, wk, _ = inputs(9, 4, 2, 128, BF, 1)
    gq, gk = w.qk_norm_rope(q, k, q_weight=wq, k_weight=wk)
    check(gq, *model(q, wq, None, None, 1e-6, False), "q")
    check(gk, *model(k, wk, None, None, 1e-6, False), "k")


def test_zero_rows_and_large_ones(w):
    q, k, wq, wk, pos = inputs(3, 4, 2, 128, BF, 1)
    q, k = q.contiguous().zero_(), (k.contiguous() * 0 + 2.0 ** 60).to(BF)
    gq, gk = w.qk_norm_rope(q, k, table(500, 128), pos, wq, wk, eps=1e-6)
    assert (gq == 0).all()
    check(gk, *model(k, wk, table(500, 128), pos, 1e-6, False), "k")


@pytest.mark.parametrize("dt", [BF, F])
def test_in_place_in_a_fused_row(w, dt):
    """In place on columns of the projection's output: the values beside them stay."""
    q, k, wq, wk, pos = inputs(19, 6, 2, 64, dt, 5, pad=8)
    base = q._base
    before = base.clone()
    cs = table(500, 64)
    want = w.qk_norm_rope(q, k, cs, pos, wq, wk)
    got = w.qk_norm_rope(q, k, cs, pos, wq, wk, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(base[:, 8 * 64:], before[:, 8 * 64:])


def test_positions_outside_leave_rows(w):
    q, k, wq, wk, pos = inputs(6, 4, 2, 128, BF, 3)
    pos[1], pos[4], pos[5] = -1, 500, 2 ** 31 - 1
    qo, ko = torch.full(q.shape, 7.0, dtype=BF, device="cuda"), torch.full(k.shape, 7.0, dtype=BF,
                                                                          device="cuda")
    cs = table(500, 128)
    w.qk_norm_rope(q, k, cs, pos, wq, wk, q_out=qo, k_out=ko)
    keep = torch.tensor([0, 2, 3], device="cuda")
    check(qo[keep], *model(q[keep], wq, cs, pos[keep], 1e-6, False), "q")
    for t in (1, 4, 5):
        assert (qo[t] == 7).all() and (ko[t] == 7).all()


def test_no_tokens_and_no_heads(w):
    q, k, wq, wk, pos = inputs(0, 4, 2, 128, BF, 3)
    gq, gk = w.qk_norm_rope(q, k, table(10, 128), pos, wq, wk)
    assert gq.shape == (0, 4, 128) and gk.shape == (0, 2, 128)
    q, k, wq, wk, pos = inputs(5, 4, 2, 128, BF, 3)
    none = torch.empty((5, 0, 128), dtype=BF, device="cuda")
    both = w.qk_norm_rope(q, k, table(500, 128), pos, wq, wk)
    assert torch.equal(w.qk_norm_rope(q, none, table(500, 128), pos, wq, wk)[0], both[0])
    assert torch.equal(w.qk_norm_rope(none, k, table(500, 128), pos, wq, wk)[1], both[1])


def test_refusals(w):
    q, k, wq, wk, pos = inputs(5, 4, 2, 128, BF, 3)
    cs = table(500, 128)
    for bad in (dict(q=q.to(F)), dict(k=k[:4]), dict(pos=pos.long()), dict(pos=pos[:4]),
                dict(wq=wq[:64]), dict(cs=cs.to(BF)), dict(cs=cs[0]), dict(q=q[..., ::2])):
        a = dict(q=q, k=k, cs=cs, pos=pos, wq=wq, wk=wk)
        a.update(bad)
        with pytest.raises((ValueError, w.W4A8Error)):
            w.qk_norm_rope(*a.values())
    with pytest.raises(w.W4A8Error):
        w.qk_norm_rope(q, k, cs, None, wq, wk)
    with pytest.raises(ValueError):
        w.qk_norm_rope(q, k, cs, pos, wq, wk, out_dtype=torch.float16)


def test_other_stream_and_graph(w):
    q, k, wq, wk, pos = inputs(40, 8, 2, 128, BF, 9)
    cs = table(500, 128)
    want = w.qk_norm_rope(q, k, cs, pos, wq, wk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = w.qk_norm_rope(q, k, cs, pos, wq, wk, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qi, ki, pi = q.clone(), k.clone(), pos.clone()
    qo, ko = torch.empty_like(qi), torch.empty_like(ki)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.qk_norm_rope(qi, ki, cs, pi, wq, wk, q_out=qo, k_out=ko)
    for seed in range(3):
        q, k, _, _, pos = inputs(40, 8, 2, 128, BF, seed)
        qi.copy_(q), ki.copy_(k), pi.copy_(pos)
        graph.replay()
        want = w.qk_norm_rope(q, k, cs, pos, wq, wk)
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])

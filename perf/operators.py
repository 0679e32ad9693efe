"""Measured cases of the row-selected operators: rows that choose experts, the
experts' products on packed 4-bit weights, and low-rank adapters beside a shared
projection.

`own` False computes the plain forms (elementary torch operations in binary32,
one rounding at the end); `own` True makes the library's calls.  `prepare` makes
the inputs from the seed, `run` is one pass through an operator, `exact` the same
outputs from the definitions in 64 bits, `work` the bytes and operations a pass
cannot do without.

Definitions (t: token, j: slot, e: expert, l: adapter)
  route    score s[t, e] = softmax over e or 1 / (1 + exp(-logit));  the key of an
           expert is s + bias[e] where there is a bias, else s, and without groups its
           logit (the score is monotone in it);  with groups, the `topk_groups` groups
           with the largest sum of their `group_top` largest keys stay;  the top_k
           experts by key, largest first, ties to the lower index;  weights[t, j] =
           s / (sum of the chosen s if renormalized) * scale.
  experts  per token: int8 codes q = rne(x * (127 / amax)), scale amax / 127;
           (g, u) = rows of W13[e] . x;  h = bf16(g / (1 + exp(-g)) * u), quantized
           per row like x;  y = W2[e] . h;  out[t] = sum_j weights[t, j] y[t, j].
           W = ch_scale * group scale * code, codes in [-7, 7], groups of 64 along K.
           Slots whose id is not an expert (-1) take no part.
  adapters out[t] = y[t] + scale[l] * B[l] . (A[l] . x[t]), l = ids[t]; -1: no adapter.
"""
import math

import torch

own = False

GROUP = 64


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a decode step: a launch's latency is all there is
        dict(name="route t1 e64", op="route", tokens=1, experts=64, top_k=8, score="softmax",
             bias=False, groups=1, topk_groups=1, group_top=1, renorm=True, dtype="bf16"),
        # a serving batch with a balance bias and limited groups
        dict(name="route t64 e256 groups", op="route", tokens=64, experts=256, top_k=8,
             score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2,
             renorm=True, dtype="f32"),
        # a prompt of ordinary length, an odd number of experts
        dict(name="route t4096 e129", op="route", tokens=4096, experts=129, top_k=6,
             score="softmax", bias=True, groups=1, topk_groups=1, group_top=1,
             renorm=False, dtype="f32"),
        # the largest prefill batch
        dict(name="route t16384 e256 groups", op="route", tokens=16384, experts=256, top_k=8,
             score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2,
             renorm=True, dtype="f32"),
        # one token of a decode step: the chosen experts' weights stream from HBM once
        dict(name="experts t1", op="experts", tokens=1, experts=64, top_k=8, hidden=2048,
             inter=768, half=False, out="bf16"),
        # a decode batch: a few rows for every expert
        dict(name="experts t16", op="experts", tokens=16, experts=32, top_k=4, hidden=4096,
             inter=2048, half=False, out="bf16"),
        # a short ragged prompt with the other half of the experts on another card: tens of
        # rows an expert, K with a trailing half chunk
        dict(name="experts t333 half", op="experts", tokens=333, experts=64, top_k=6,
             hidden=2112, inter=1088, half=True, out="f32"),
        # a prompt over few large experts (the feed-forward sizes of the prefill workload)
        dict(name="experts t4096 large", op="experts", tokens=4096, experts=8, top_k=2,
             hidden=4096, inter=14336, half=False, out="bf16"),
        # a prompt over many middle-sized experts
        dict(name="experts t4096 many", op="experts", tokens=4096, experts=32, top_k=4,
             hidden=4096, inter=1408, half=False, out="bf16"),
        # a decode step of few requests beside the decode workload's projection
        dict(name="adapters t8", op="adapters", tokens=8, adapters=8, rank=16, k=4096, n=4096,
             segments=False, out="bf16"),
        # a full decode batch with an adapter for every other request, high rank
        dict(name="adapters t64", op="adapters", tokens=64, adapters=32, rank=64, k=4096,
             n=14336, segments=False, out="bf16"),
        # prompts of several requests in one batch beside the FFN-down projection
        dict(name="adapters t2047", op="adapters", tokens=2047, adapters=6, rank=32, k=28672,
             n=8192, segments=True, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        # 3072 is no size of this repository's workloads, as a gate-up width neither
        if 3072 not in c.values() and 2 * c.get("inter", 0) != 3072:
            return c


def _draw(rng):
    op = rng.choice(["route", "experts", "adapters"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * rng.randint(max(2, 8 // groups), 256 // groups)
        topk_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(8, topk_groups * (experts // groups)))
        return dict(op="route", tokens=_log_int(rng, 1, 16384), experts=experts, top_k=top_k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6,
                    groups=groups, topk_groups=topk_groups, group_top=rng.randint(1, 2),
                    renorm=rng.random() < 0.7,
                    dtype=rng.choice(["f32", "bf16"]))
    if op == "experts":
        while True:
            experts = rng.randint(4, 96)
            tokens, top_k = _log_int(rng, 1, 4096), rng.randint(1, min(8, experts))
            c = dict(op="experts", tokens=tokens, experts=experts, top_k=top_k,
                     hidden=64 * rng.randint(16, 64), inter=64 * _log_int(rng, 4, 224),
                     half=tokens * top_k >= 16 and rng.random() < 0.25,
                     out=rng.choice(["bf16", "bf16", "f32"]))
            # no more weights and no more products than the largest listed case
            if (c["experts"] * c["hidden"] * c["inter"] <= 8 * 4096 * 14336 and
                    c["tokens"] * c["top_k"] * c["hidden"] * c["inter"] <=
                    4096 * 2 * 4096 * 14336):
                return c
    while True:
        tokens = _log_int(rng, 1, 4096)
        c = dict(op="adapters", tokens=tokens, adapters=rng.randint(1, 48),
                 rank=rng.choice([8, 16, 16, 32, 64, 128]), k=8 * _log_int(rng, 128, 3584),
                 n=8 * _log_int(rng, 128, 1792), segments=tokens > 64,
                 out=rng.choice(["bf16", "bf16", "f32"]))
        if (c["tokens"] * (c["k"] + 2 * c["n"]) <= 2047 * (28672 + 4 * 8192) and
                c["adapters"] * c["rank"] * (c["k"] + c["n"]) <= 32 * 64 * (4096 + 14336)):
            return c


# ----------------------------------------------------------------- inputs --

def _rand(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


def _router_logits(tokens, experts, gen):
    """Logits of a trained router: per-token spread plus a popularity of the experts."""
    return 1.5 * _rand((tokens, experts), gen) + 0.5 * _rand((experts,), gen)


def _pack(q, s):
    """Codes q int8 [N, K] in [-7, 7] and group scales s uint8 [N, K / 64] -> the packed
    weight layout: tiles of 16 channels, chunks of 128 along K (the last one 64 wide if
    K % 128 == 64), a 16-byte (8-byte) record per lane = channel + 16 (k % 64 / 16)."""
    n, k = q.shape
    t, full = n // 16, k // 128
    u = (q + 8).to(torch.uint8).view(t, 16, k)
    parts = []
    if full:
        v = u[:, :, :full * 128].reshape(t, 16, full, 2, 4, 2, 2, 4)
        v = v.permute(0, 2, 4, 1, 3, 5, 6, 7)             # t, chunk, kq, c, step, half, hi, byte
        parts.append((v[..., 0, :] | (v[..., 1, :] << 4)).reshape(t, full * 1024))
    if k % 128:
        v = u[:, :, full * 128:].reshape(t, 16, 4, 2, 2, 4).permute(0, 2, 1, 3, 4, 5)
        parts.append((v[..., 0, :] | (v[..., 1, :] << 4)).reshape(t, 512))
    packed = torch.cat(parts, 1).reshape(-1).contiguous()
    return packed, s.view(t, 16, k // GROUP).permute(0, 2, 1).reshape(-1).contiguous()


def _weights(experts, n, k, gen):
    """Stacked experts' weights [experts, n, k]: codes, group scales and channel scales as
    two-level quantization of normal weights of deviation 0.02 gives them, and the packed
    form."""
    rows = experts * n
    q = torch.empty((rows, k), dtype=torch.int8, device=gen.device)
    for r in range(0, rows, 8192):
        q[r:r + 8192] = (2.7 * _rand((min(8192, rows - r), k), gen)).round_().clamp_(-7, 7)
    s = torch.randint(7, 14, (rows, k // GROUP), generator=gen, device=gen.device,
                      dtype=torch.uint8)
    c = 7.5e-4 * (1 + 0.1 * _rand((rows,), gen)).clamp_(0.5, 1.5)
    packed, grp = _pack(q, s)
    return dict(q=q.view(experts, n, k), s=s.view(experts, n, k // GROUP),
                c=c.view(experts, n), packed=(packed, grp, c))


def prepare(case, seed):
    gen = torch.Generator(device=_dev())
    gen.manual_seed(1000003 * int(seed) + 17)
    st = dict(case=case)
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        st["logits"] = _router_logits(t, e, gen).to(
            torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        st["bias"] = 0.1 * _rand((e,), gen) if case["bias"] else None
    elif case["op"] == "experts":
        t, e, h, i = (case[x] for x in ("tokens", "experts", "hidden", "inter"))
        st["x"] = _rand((t, h), gen).to(torch.bfloat16)
        # half: as many experts again are on another card, their slots are not ours (-1)
        p = torch.softmax(_router_logits(t, 2 * e if case["half"] else e, gen), 1)
        w, ids = torch.sort(p, dim=1, descending=True, stable=True)
        ids = ids[:, :case["top_k"]].to(torch.int32)
        st["ids"] = torch.where(ids < e, ids, -1).contiguous()
        w = w[:, :case["top_k"]]
        st["weights"] = (w / w.sum(1, keepdim=True)).contiguous()
        st["w13"] = _weights(e, 2 * i, h, gen)              # per expert: gate rows, then up rows
        st["w2"] = _weights(e, h, i, gen)
    else:
        t, a, r, k, n = (case[x] for x in ("tokens", "adapters", "rank", "k", "n"))
        st["x"] = _rand((t, k), gen).to(torch.bfloat16)
        st["y"] = _rand((t, n), gen).to(torch.bfloat16 if case["out"] == "bf16"
                                        else torch.float32)
        st["a"] = (_rand((a, r, k), gen) * k ** -0.5).to(torch.bfloat16)
        st["b"] = (_rand((a, n, r), gen) * (0.5 * r ** -0.5)).to(torch.bfloat16)
        st["scale"] = 0.5 + 1.5 * torch.rand((a,), generator=gen, device=gen.device)
        if case["segments"]:    # prompts of several requests, one after the other
            cuts = torch.sort(torch.randint(0, t + 1, (2 * a,), generator=gen,
                                            device=gen.device)).values
            req = torch.searchsorted(cuts, torch.arange(t, device=gen.device), right=True)
            of = torch.randint(-1, a, (2 * a + 1,), generator=gen, device=gen.device)
            st["ids"] = of[req].to(torch.int32).contiguous()
        else:                   # one row a request, an eighth of them without an adapter
            ids = torch.randint(0, a, (t,), generator=gen, device=gen.device)
            none = torch.rand((t,), generator=gen, device=gen.device) < 0.125
            st["ids"] = torch.where(none, -1, ids).to(torch.int32).contiguous()
    return st


# ------------------------------------------------------------ plain forms --

def _top(keys, count):
    """Indices of the `count` largest keys of each row, largest first, ties to the lower."""
    return torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :count]


def _plain_route(st):
    c = st["case"]
    x = st["logits"].float()
    if c["score"] == "softmax":
        p = torch.exp(x - x.max(1, keepdim=True).values)
        # summed so that no order of the terms shows in the rounded total
        s = p / p.sum(1, keepdim=True, dtype=torch.float64).float()
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    key = s + st["bias"] if st["bias"] is not None else s if c["groups"] > 1 else x
    if c["groups"] > 1:
        t, per = x.shape[0], c["experts"] // c["groups"]
        best = torch.sort(key.view(t, c["groups"], per), dim=2, descending=True).values
        keep = torch.zeros((t, c["groups"]), dtype=torch.bool, device=x.device)
        keep.scatter_(1, _top(best[..., :c["group_top"]].sum(2), c["topk_groups"]), True)
        key = torch.where(keep.repeat_interleave(per, 1), key, float("-inf"))
    ids = _top(key, c["top_k"])
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w * _scale(c)


def _scale(c):
    return 2.5 if c["groups"] > 1 else 1.0


def _quant(x):
    """Per-row int8 codes (as binary32) and scales of x (binary32)."""
    amax = x.abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, 127.0 / amax, 0.0)
    return torch.clamp(torch.round(x * inv), -127, 127), amax / 127.0


def _places(ids, groups):
    """For rows with an id in [0, groups): the row's place in [groups, most], and most."""
    hot = (ids[:, None] == torch.arange(groups, device=ids.device)).int()
    rank = (hot.cumsum(0) - 1).gather(1, ids.clamp_min(0).long()[:, None])[:, 0]
    most = max(1, int(hot.sum(0).max()))
    return ids.long() * most + rank, most


def _grouped(rows, place, used, groups, most, w_t):
    """rows [R, K] times the weights [groups, K, N] of each used row's group -> [R, N]."""
    pad = torch.zeros((groups * most, rows.shape[1]), device=rows.device)
    pad[place[used]] = rows[used]
    y = torch.bmm(pad.view(groups, most, -1), w_t).view(groups * most, -1)
    out = torch.zeros((rows.shape[0], y.shape[1]), device=rows.device)
    out[used] = y[place[used]]
    return out


def _plain_experts(st):
    c = st["case"]
    t, k, i = c["tokens"], c["top_k"], c["inter"]
    ids = st["ids"].reshape(-1)
    used = (ids >= 0).nonzero()[:, 0]
    met, of = torch.unique(ids[used], return_inverse=True)     # the experts that have rows
    met = met.long()
    if not len(met):
        return torch.zeros(st["x"].shape, device=ids.device,
                           dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    local = torch.full_like(ids, -1)
    local[used] = of.to(ids.dtype)
    place, most = _places(local, len(met))

    def product(q, scale, w):
        # whole numbers below 2^24 all along: the sums are exact, the scales come after
        deq = w["q"][met].float() * w["s"][met].float().repeat_interleave(GROUP, 2)
        acc = _grouped(q, place, used, len(met), most, deq.transpose(1, 2).contiguous())
        return acc * scale * w["c"][ids.clamp_min(0).long()]

    q, s = _quant(st["x"].float())
    gu = product(q.repeat_interleave(k, 0), s.repeat_interleave(k, 0), st["w13"])
    g, u = gu[:, :i], gu[:, i:]
    h = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16).float()
    q, s = _quant(h)
    y = product(q, s, st["w2"])
    out = (y.view(t, k, -1) * st["weights"][..., None]).sum(1)
    return out.to(torch.bfloat16) if c["out"] == "bf16" else out


def _plain_adapters(st):
    c = st["case"]
    ids = st["ids"]
    used = (ids >= 0).nonzero()[:, 0]
    place, most = _places(ids, c["adapters"])
    v = _grouped(st["x"].float(), place, used, c["adapters"], most,
                 st["a"].float().transpose(1, 2).contiguous())
    d = _grouped(v, place, used, c["adapters"], most,
                 st["b"].float().transpose(1, 2).contiguous())
    scale = torch.where(ids >= 0, st["scale"][ids.clamp_min(0).long()], 0.0)
    return (st["y"].float() + scale[:, None] * d).to(st["y"].dtype)


def run(state):
    c = state["case"]
    if own:
        from w4a8_quantized_gemm_quantize_amd import binding
        if c["op"] == "route":
            return binding.moe_route(state["logits"], c["top_k"], bias=state["bias"],
                                     score=c["score"], groups=c["groups"],
                                     topk_groups=c["topk_groups"], group_top=c["group_top"],
                                     renormalize=c["renorm"], scale=_scale(c))
        if c["op"] == "experts":
            return binding.w4a8_moe_ffn(state["x"], state["ids"], state["weights"],
                                        state["w13"]["packed"], state["w2"]["packed"],
                                        c["inter"], out_dtype=torch.bfloat16
                                        if c["out"] == "bf16" else torch.float32)
        return binding.lora_add(state["x"], state["a"], state["b"], state["ids"], state["y"],
                                scale=state["scale"])
    if c["op"] == "route":
        return _plain_route(state)
    if c["op"] == "experts":
        return _plain_experts(state)
    return _plain_adapters(state)


# -------------------------------------------------------- 64-bit reference --

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "route":
        x = st["logits"].to(f64)
        s = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
        key = s if st["bias"] is None and case["groups"] > 1 else x
        if st["bias"] is not None:
            key = s + st["bias"].to(f64)
        if case["groups"] > 1:
            per = case["experts"] // case["groups"]
            best = torch.topk(key.view(len(x), case["groups"], per), case["group_top"], 2)
            order = torch.argsort(best.values.sum(2), dim=1, descending=True, stable=True)
            drop = order[:, case["topk_groups"]:]
            member = torch.arange(case["experts"], device=x.device) // per
            lost = (member[None, :, None] == drop[:, None, :]).any(2)
            key = key.masked_fill(lost, -math.inf)
        ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["top_k"]]
        w = torch.take_along_dim(s, ids, 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        # an expert is a choice among near equals: no value in 64 bits
        return None, w * (2.5 if case["groups"] > 1 else 1.0)

    def codes(v):
        # the definition's codes come from binary32 products of bf16 values (a code at a
        # half goes where that product rounds); all that follows is in 64 bits
        v = v.float()
        top = v.abs().amax(1, keepdim=True)
        inverse = torch.where(top > 0, 127 / top, 0.0)
        return torch.round(v * inverse).to(f64), top.to(f64) / 127

    if case["op"] == "experts":
        ids = st["ids"].long()
        out = torch.zeros((case["tokens"], case["hidden"]), dtype=f64, device=ids.device)
        q, s = codes(st["x"])
        i = case["inter"]
        for e in range(case["experts"]):
            tok, slot = (ids == e).nonzero(as_tuple=True)
            if not len(tok):
                continue

            def dense(w):
                g = w["s"][e].to(f64)[:, :, None] * w["c"][e].to(f64)[:, None, None]
                return (w["q"][e].to(f64).view(len(g), -1, GROUP) * g).view(len(g), -1)

            gu = (q[tok] @ dense(st["w13"]).T) * s[tok]
            h = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
            hq, hs = codes(h.to(torch.bfloat16))
            y = (hq @ dense(st["w2"]).T) * hs
            out.index_put_((tok,), y * st["weights"][tok, slot].to(f64)[:, None],
                           accumulate=True)
        return out
    out = st["y"].to(f64)
    for a in range(case["adapters"]):
        rows = (st["ids"] == a).nonzero()[:, 0]
        if len(rows):
            v = st["x"][rows].to(f64) @ st["a"][a].to(f64).T
            out[rows] += st["scale"][a].to(f64) * (v @ st["b"][a].to(f64).T)
    return out


# ------------------------------------------------------------------- work --

def _met(choices, among):
    """Expected number of different ones among `among` after so many even choices."""
    return among * (1 - (1 - 1 / among) ** choices)


def work(case):
    t = case["tokens"]
    if case["op"] == "route":
        e, k = case["experts"], case["top_k"]
        size = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=t * e * size + (4 * e if case["bias"] else 0) + t * k * 8,
                    flops=4 * t * e)
    if case["op"] == "experts":
        e, k, h, i = (case[x] for x in ("experts", "top_k", "hidden", "inter"))
        share = 0.5 if case["half"] else 1.0
        met = e * (1 - (1 - share * k / e) ** t)
        per = 3 * h * i * (0.5 + 1 / GROUP) + 4 * (2 * i + h)
        return dict(bytes=met * per + t * h * (2 + (2 if case["out"] == "bf16" else 4)) +
                    t * k * 8, flops=6 * t * k * share * h * i)
    a, r, k, n = (case[x] for x in ("adapters", "rank", "k", "n"))
    size = 2 if case["out"] == "bf16" else 4
    # of the prompts' 2 a + 1 segments one in a + 1 has no adapter, of single rows one in 8
    met = _met((2 * a + 1) * a / (a + 1), a) if case["segments"] else _met(t * 0.875, a)
    return dict(bytes=t * (2 * k + 2 * n * size + 4) + met * r * (k + n) * 2,
                flops=2 * t * r * (k + n))

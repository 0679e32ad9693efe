"""Measured cases of the attention half of a served transformer block: norms and
rotation of queries and keys, the paged 8-bit cache they are written to and read from,
and attention over that cache.

`own` False computes the plain forms (elementary torch operations in binary32, one
rounding at the end); `own` True makes the library's calls.  `prepare` makes the inputs
from the seed, `run` is one pass through an operator, `exact` the same outputs from the
definitions in 64 bits, `work` the bytes and operations a pass cannot do without.

Definitions (t: row, h: head, d: element of a head, s: sequence)
  rope    y = x * w[d] / sqrt(mean over d of x^2 + eps); the first `rot` elements turn in
          pairs (a, b): (a c - b s, b c + a s) with c, s the cosine and sine of the row's
          position; pairs are (j, j + rot / 2), or (2 j, 2 j + 1) where interleaved.
  store   rows of a sequence are its last ones: row i of n is token len - n + i.  Per page,
          head, and keys and values apart: scale = max |x| / 127 over the page's new tokens;
          a page that holds older tokens keeps its scale unless the new one is larger, and
          then their codes become rne(code * (old scale / new scale)).  Codes are
          rne(x * (1 / scale)) within 127.  Read back: code * scale, of all tokens of the
          pages written to.
  read    code * scale of the whole sequences.
  attn    row i of n sits at p = len - n + i and sees the tokens j < len with j <= p, and
          j > p - window where there is a window.  out = softmax(scale * q . k_j) . v_j and
          lse, the logarithm of the softmax's sum; query head h reads head h / (q_heads /
          kv_heads) of the cache.
"""
import math

import torch

own = False


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ------------------------------------------------------------------ cases --

def _rope(name, tokens, q_heads, kv_heads, dim, rot, interleaved, dtype, out):
    return dict(name=name, op="rope", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                rot=rot, interleaved=interleaved, dtype=dtype, out=out)


def _store(name, seqs, rows, uneven, before, kv_heads, dim, page, dtype):
    return dict(name=name, op="store", seqs=seqs, rows=rows, uneven=uneven, before=before,
                kv_heads=kv_heads, dim=dim, page=page, dtype=dtype)


def _read(name, seqs, tokens, kv_heads, dim, page, out):
    return dict(name=name, op="read", seqs=seqs, tokens=tokens, kv_heads=kv_heads, dim=dim,
                page=page, out=out)


def _attn(name, seqs, rows, uneven, before, q_heads, kv_heads, dim, page, window=0):
    return dict(name=name, op="attn", seqs=seqs, rows=rows, uneven=uneven, before=before,
                q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page, window=window)


def listed():
    return [
        # one token of a decode step: a launch's latency is all there is
        _rope("rope t1", 1, 32, 8, 128, 128, False, "bf16", "bf16"),
        # a short prompt of a model that turns a third of each head, pairs side by side, from a
        # projection that left binary32
        _rope("rope t333 partial", 333, 14, 2, 96, 32, True, "f32", "bf16"),
        # a prefill batch
        _rope("rope t8192", 8192, 64, 8, 128, 128, False, "bf16", "bf16"),
        # a decode step of a full batch: one token a sequence, into pages partly filled
        _store("store t64 decode", 64, 64, False, 700, 8, 128, 16, "bf16"),
        # prompts of ragged lengths that continue cached prefixes
        _store("store t8191 prompts", 5, 8191, True, 37, 8, 128, 64, "bf16"),
        # a few short sequences, to be handed to another process
        _read("read t1500", 3, 1500, 4, 64, 32, "f32"),
        # a batch's whole cache
        _read("read t65536", 8, 65536, 8, 128, 16, "bf16"),
        # one request's decode step with a short past: latency
        _attn("attn t1", 1, 1, False, 500, 32, 8, 128, 16),
        # a full decode batch: the cache streams from HBM once
        _attn("attn t64 decode", 64, 64, False, 8192, 64, 8, 128, 16),
        # three long sequences, three proposed tokens each: few rows, a long axis
        _attn("attn t9 long", 3, 9, False, 110000, 40, 8, 128, 128),
        # prompts of ragged lengths without a past: the matrix cores
        _attn("attn t8191 prompts", 2, 8191, True, 0, 64, 8, 128, 64),
        # a chunk of a long prompt, narrow heads, seven query heads a cache head
        _attn("attn t500 chunk", 1, 500, False, 30000, 28, 4, 64, 32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        del c["name"]
        if _cost(c):
            return c


_DIMS = [64, 96, 128, 128, 128, 192, 256]


def _draw(rng):
    op = rng.choice(["rope", "store", "read", "attn", "attn"])
    kv_heads, dim, page = rng.randint(1, 8), rng.choice(_DIMS), rng.choice([16, 32, 64, 128])
    if op == "rope":
        rot = rng.choice([dim, dim, dim // 2, 32])
        return _rope("", _log_int(rng, 1, 8192), kv_heads * rng.randint(1, 8), kv_heads, dim, rot,
                     rng.random() < 0.3, rng.choice(["bf16", "bf16", "f32"]),
                     rng.choice(["bf16", "bf16", "f32"]))
    if op == "store":
        seqs = _log_int(rng, 1, 64)
        rows = seqs * _log_int(rng, 1, 4096)
        return _store("", seqs, rows, rows > 8 * seqs, _log_int(rng, 1, 2000) - 1, kv_heads, dim,
                      page, rng.choice(["bf16", "bf16", "f32"]))
    if op == "read":
        return _read("", _log_int(rng, 1, 32), _log_int(rng, 32, 65536), kv_heads, dim, page,
                     rng.choice(["bf16", "f32"]))
    group = rng.randint(1, 8)
    if rng.random() < 0.5:          # a token or a few for every sequence
        seqs = _log_int(rng, 1, 64)
        return _attn("", seqs, seqs * rng.choice([1, 1, 1, 2, 3, 5]), False,
                     _log_int(rng, 16, 110000), kv_heads * group, kv_heads, dim, page,
                     rng.choice([0, 0, 0, 1000]))
    seqs = rng.randint(1, 6)        # prompts, or chunks of them
    return _attn("", seqs, seqs * _log_int(rng, 10, 8191), True,
                 rng.choice([0, 0, _log_int(rng, 16, 30000)]), kv_heads * group, kv_heads, dim,
                 page, rng.choice([0, 0, 0, 1000]))


def _cost(c):
    """Whether a drawn case takes no more than the largest listed ones."""
    w = work(c)
    if c["op"] == "rope":
        return True
    if c["op"] in ("store", "read"):
        return w["bytes"] <= 4.2e8
    _, lens, rows = _lengths(c)
    grid = c["seqs"] * c["q_heads"] * max(rows) * max(lens)       # the plain form's scores
    return w["bytes"] <= 1.1e9 and w["flops"] <= 5.9e11 and grid <= 3.4e9


# ---------------------------------------------------------------- lengths --

def _spread(total, parts, uneven):
    """`total` in `parts` whole numbers: even, or from about a half to about twice the mean."""
    weights = [0.5 + (0.618 * (i + 1)) % 1.0 * 1.5 if uneven else 1.0 for i in range(parts)]
    whole = sum(weights)
    ends = [round(total * sum(weights[:i + 1]) / whole) for i in range(parts)]
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def _lengths(c):
    """Of each sequence: tokens before the rows, tokens in all, rows."""
    n = c["seqs"]
    if c["op"] == "read":
        lens = _spread(c["tokens"], n, True)
        return [0] * n, lens, lens
    rows = _spread(c["rows"], n, c["uneven"])
    past = _spread(c["before"] * n, n, True) if c["before"] else [0] * n
    return past, [a + b for a, b in zip(past, rows)], rows


# ----------------------------------------------------------------- inputs --

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rand(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _pack(codes):
    """Codes int8 [..., page, dim] of keys -> the cache's layout (bytes hold code + 128): tiles
    of 16 tokens, chunks of 64 elements (the last one 32 wide where dim % 64 == 32), a 16-byte
    (8-byte) record per lane = token + 16 (element % 64 / 16)."""
    *lead, page, dim = codes.shape
    u = (codes.to(torch.int16) + 128).to(torch.uint8).view(-1, page // 16, 16, dim)
    full = dim // 64 * 64
    # n, tile, token, chunk, quarter, element -> n, tile, chunk, quarter, token, element
    parts = [u[..., :full].reshape(*u.shape[:3], full // 64, 4, 16).permute(0, 1, 3, 4, 2, 5)
             .reshape(*u.shape[:2], full * 16)]
    if dim % 64:
        parts.append(u[..., full:].reshape(*u.shape[:3], 4, 8).permute(0, 1, 3, 2, 4)
                     .reshape(*u.shape[:2], 32 * 16))
    return torch.cat(parts, 2).view(*lead, page, dim)


def _pack_values(codes):
    """The same for values: lane = element % 16 + 16 (token / 4), and a record holds four
    tokens of each of the chunk's four (two) elements with that remainder."""
    *lead, page, dim = codes.shape
    u = (codes.to(torch.int16) + 128).to(torch.uint8).view(-1, page // 16, 4, 4, dim)
    full = dim // 64 * 64
    # n, tile, quad, token, chunk, sixteenth, element -> n, tile, chunk, quad, element, 16th, token
    parts = [u[..., :full].reshape(*u.shape[:4], full // 64, 4, 16).permute(0, 1, 4, 2, 6, 5, 3)
             .reshape(*u.shape[:2], full * 16)]
    if dim % 64:
        parts.append(u[..., full:].reshape(*u.shape[:4], 2, 16).permute(0, 1, 2, 5, 4, 3)
                     .reshape(*u.shape[:2], 32 * 16))
    return torch.cat(parts, 2).view(*lead, page, dim)


def _cache(case, lens, gen):
    """A pool of pages in use by sequences of these lengths, pages in any order: block table,
    codes of normal keys and values, scales, and the packed form."""
    h, dim, page, n = case["kv_heads"], case["dim"], case["page"], len(lens)
    need = [-(-x // page) for x in lens]
    pages = sum(need) + 3                                  # a few that nobody uses
    order = torch.randperm(pages, generator=gen, device=gen.device).to(torch.int32)
    table = torch.full((n, max(max(need), 1)), -1, dtype=torch.int32, device=gen.device)
    at = torch.arange(table.shape[1], device=gen.device)[None] < _ints(need, gen.device)[:, None]
    table[at] = order[:sum(need)]
    codes = torch.empty((2, pages, h, page, dim), dtype=torch.int8, device=gen.device)
    flat = codes.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_((33.0 * _rand((part.numel(),), gen)).round_().clamp_(-127, 127))
    sigma = 0.5 + torch.rand((1, h, 2), generator=gen, device=gen.device)
    scales = sigma * (0.8 + 0.4 * torch.rand((pages, h, 2), generator=gen, device=gen.device)) / 33
    kv = torch.stack([_pack(codes[0]), _pack_values(codes[1])], 2).contiguous()
    return dict(table=table, codes=codes, scales=scales, plain_scales=scales.clone(), kv=kv)


def _angles(tokens, rot, gen):
    """A table of cosines and sines over positions, and each row's position: a stretch of a
    long prompt and single rows far apart."""
    most = 40000
    freq = 1e6 ** (-torch.arange(rot // 2, device=gen.device, dtype=torch.float64) / (rot // 2))
    angle = torch.arange(most, device=gen.device, dtype=torch.float64)[:, None] * freq
    table = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    start = int(torch.randint(0, most - tokens, (1,), generator=gen, device=gen.device))
    pos = torch.arange(start, start + tokens, device=gen.device)
    far = torch.rand((tokens,), generator=gen, device=gen.device) < 0.2
    other = torch.randint(0, most, (tokens,), generator=gen, device=gen.device)
    return table, torch.where(far, other, pos).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=_dev())
    gen.manual_seed(1000003 * int(seed) + 29)
    st = dict(case=case)
    dim, h = case["dim"], case["kv_heads"]
    if case["op"] == "rope":
        t, hq, dt = case["tokens"], case["q_heads"], _TYPES[case["dtype"]]
        # the projection's rows: queries, keys, values side by side
        rows = (_rand((t, (hq + 2 * h) * dim), gen) *
                (0.5 + torch.rand((t, 1), generator=gen, device=gen.device))).to(dt)
        st["q"] = rows[:, :hq * dim].view(t, hq, dim)
        st["k"] = rows[:, hq * dim:(hq + h) * dim].view(t, h, dim)
        st["wq"] = 1 + 0.2 * _rand((dim,), gen)
        st["wk"] = 1 + 0.2 * _rand((dim,), gen)
        st["angles"], st["pos"] = _angles(t, case["rot"], gen)
        return st
    past, lens, rows = _lengths(case)
    st.update(_cache(case, lens, gen), lens=_ints(lens, gen.device))
    starts = [sum(rows[:i]) for i in range(len(rows) + 1)]
    st["starts"], st["rows"], st["most_rows"] = _ints(starts, gen.device), starts[-1], max(rows)
    st["most_len"] = max(lens)
    if case["op"] == "store":
        dt = _TYPES[case["dtype"]]
        kv = _rand((starts[-1], 2 * h * dim), gen)
        # about one new row in four is the largest of its page
        kv *= 2.5 * torch.rand((starts[-1], 1), generator=gen, device=gen.device)
        kv = kv.to(dt)
        st["k"] = kv[:, :h * dim].view(-1, h, dim)
        st["v"] = kv[:, h * dim:].view(-1, h, dim)
        # what the pages written to hold afterwards: older tokens of the first one, and the rows
        held = [p % case["page"] + n if n else 0 for p, n in zip(past, rows)]
        ends = [sum(held[:i]) for i in range(len(held) + 1)]
        st["held"], st["held_rows"] = _ints(ends, gen.device), ends[-1]
        st["most_held"] = max(held)
    elif case["op"] == "attn":
        st["q"] = _rand((starts[-1], case["q_heads"] * dim), gen).to(torch.bfloat16) \
            .view(-1, case["q_heads"], dim)
    return st


# ------------------------------------------------------------ plain forms --

def _plain_rope(st):
    c = st["case"]
    rot, half = c["rot"], c["rot"] // 2
    angle = st["angles"][st["pos"].long()][:, None]
    cos, sin = angle[..., :half], angle[..., half:]

    def turned(x, w):
        x = x.float()
        y = x * (torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6) * w)
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
        else:
            a, b = y[..., :half], y[..., half:rot]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
        return torch.cat([z, y[..., rot:]], 2).to(_TYPES[c["out"]])

    return turned(st["q"], st["wq"]), turned(st["k"], st["wk"])


def _owner(starts, rows):
    """The sequence of each of `rows` rows, and its place there."""
    row = torch.arange(rows, device=starts.device)
    seq = torch.searchsorted(starts[1:].long(), row, right=True)
    return seq, row - starts[seq].long()


def _token_values(st, starts, rows):
    """Codes times scales of the last starts[s + 1] - starts[s] tokens of each sequence, in
    binary32: [2, rows, heads, dim]."""
    page = st["case"]["page"]
    seq, i = _owner(starts, rows)
    at = st["lens"][seq].long() - (starts[seq + 1] - starts[seq]).long() + i
    block = st["table"][seq, at // page].long()
    codes = st["codes"][:, block, :, at % page].transpose(0, 1)    # from rows, 2, heads, dim
    return codes.float() * st["plain_scales"][block].permute(2, 0, 1)[..., None]


def _plain_store(st):
    c = st["case"]
    page, rows, scales = c["page"], st["rows"], st["plain_scales"]
    seq, i = _owner(st["starts"], rows)
    first = (st["lens"] - (st["starts"][1:] - st["starts"][:-1])).long()
    at = first[seq] + i
    block = st["table"][seq, at // page].long()
    x = torch.stack([st["k"], st["v"]]).float()            # 2, rows, heads, dim
    top = x.abs().amax(3).permute(1, 2, 0)                 # rows, heads, 2
    most = torch.zeros_like(scales).scatter_reduce(
        0, block[:, None, None].expand_as(top), top, "amax")
    new = most / torch.full_like(most, 127.0)
    # pages with older tokens: the first row's, where it does not start a page
    older = (st["starts"][1:] > st["starts"][:-1]) & (first % page > 0)
    kept = first[older] % page
    old = st["table"][older, first[older] // page].long()
    was = scales[old]
    now = torch.maximum(was, new[old])
    ratio = torch.where(now > was, was / now, 1.0).permute(2, 0, 1)[..., None, None]
    older_token = (torch.arange(page, device=old.device) < kept[:, None])[None, :, None, :, None]
    codes = st["codes"][:, old].float()
    codes = torch.where(older_token, torch.round(codes * ratio), codes)
    st["codes"][:, old] = codes.to(torch.int8)
    scales[block] = new[block]
    scales[old] = now
    scale = scales[block].permute(2, 0, 1)[..., None]
    inverse = torch.where(scale > 0, torch.ones_like(scale) / scale, 0.0)
    q = torch.clamp(torch.round(x * inverse), -127, 127).to(torch.int8)
    st["codes"][:, block, :, at % page] = q.transpose(0, 1)
    got = _token_values(st, st["held"], st["held_rows"])
    return got[0], got[1]


def _plain_read(st):
    got = _token_values(st, st["starts"], st["rows"]).to(_TYPES[st["case"]["out"]])
    return got[0], got[1]


def _plain_attn(st):
    c = st["case"]
    h, dim, page, n, length = c["kv_heads"], c["dim"], c["page"], st["most_rows"], st["most_len"]
    group, seqs = c["q_heads"] // h, c["seqs"]
    table = st["table"].clamp_min(0).long()

    def dense(i):                                          # seqs, heads, tokens, dim
        x = st["codes"][i][table].permute(0, 2, 1, 3, 4).float()
        x = x * st["plain_scales"][table][..., i].transpose(1, 2)[..., None, None]
        return x.reshape(seqs * h, -1, dim)[:, :length].contiguous()

    seq, i = _owner(st["starts"], st["rows"])
    q = torch.zeros((seqs, n, c["q_heads"], dim), device=seq.device)
    q[seq, i] = st["q"].float()
    q = q.view(seqs, n, h, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs * h, group * n, dim)
    scores = torch.bmm(q * dim ** -0.5, dense(0).transpose(1, 2).contiguous())
    scores = scores.view(seqs, h, group, n, length)
    lens = st["lens"].long()
    count = (st["starts"][1:] - st["starts"][:-1]).long()
    p = (lens - count)[:, None, None] + torch.arange(n, device=seq.device)[None, :, None]
    j = torch.arange(length, device=seq.device)[None, None]
    seen = (j <= p) & (j < lens[:, None, None])
    if c["window"]:
        seen &= j > p - c["window"]
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(4, keepdim=True)
    e = scores.sub_(torch.where(top > float("-inf"), top, 0.0)).exp_()
    total = e.sum(4)
    out = torch.bmm(e.view(seqs * h, group * n, length), dense(1)).view(seqs, h, group, n, dim)
    out = out / total[..., None]
    lse = top[..., 0] + torch.log(total)
    out = out.permute(0, 3, 1, 2, 4).reshape(seqs, n, c["q_heads"], dim)[seq, i]
    lse = lse.permute(0, 3, 1, 2).reshape(seqs, n, c["q_heads"])[seq, i]
    return out.to(torch.bfloat16), lse


def run(state):
    c = state["case"]
    if own:
        from w4a8_quantized_gemm_quantize_amd import binding
        if c["op"] == "rope":
            return binding.qk_norm_rope(state["q"], state["k"], state["angles"], state["pos"],
                                        q_weight=state["wq"], k_weight=state["wk"], eps=1e-6,
                                        interleaved=c["interleaved"], out_dtype=_TYPES[c["out"]])
        if c["op"] == "attn":
            return binding.attn_kv8(state["q"], state["kv"], state["scales"], state["table"],
                                    state["lens"], state["starts"], max_rows=state["most_rows"],
                                    window=c["window"], want_lse=True)
        if c["op"] == "store":
            binding.kv8_write(state["k"], state["v"], state["kv"], state["scales"],
                              state["table"], state["lens"], state["starts"])
            return binding.kv8_read(state["kv"], state["scales"], state["table"], state["lens"],
                                    state["held"], tokens=state["held_rows"],
                                    out_dtype=torch.float32)
        return binding.kv8_read(state["kv"], state["scales"], state["table"], state["lens"],
                                state["starts"], tokens=state["rows"],
                                out_dtype=_TYPES[c["out"]])
    if c["op"] == "rope":
        return _plain_rope(state)
    if c["op"] == "store":
        return _plain_store(state)
    if c["op"] == "read":
        return _plain_read(state)
    return _plain_attn(state)


# -------------------------------------------------------- 64-bit reference --

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "rope":
        rot = case["rot"]
        first = torch.arange(0, rot, 2) if case["interleaved"] else torch.arange(rot // 2)
        second = first + (1 if case["interleaved"] else rot // 2)
        angle = st["angles"].to(f64).index_select(0, st["pos"].long()).unsqueeze(1)
        turn = torch.complex(*angle.split(rot // 2, 2))
        outs = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            x = x.to(f64)
            y = x * w.to(f64) / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6)
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            outs.append(y)
        return tuple(outs)
    page, dim, h = case["page"], case["dim"], case["kv_heads"]
    _, lens, rows = _lengths(case)
    table = st["table"].long()

    def tokens(i, s, lo, hi):       # values of sequence s's tokens lo .. hi - 1: hi - lo, h, dim
        used = table[s, lo // page:-(-hi // page)]
        v = st["codes"][i][used].to(f64) * st["plain_scales"][used][..., i].to(f64)[..., None, None]
        v = v.transpose(1, 2).reshape(-1, h, dim)
        return v[lo % page:lo % page + hi - lo]

    if case["op"] == "read":
        return tuple(torch.cat([tokens(i, s, 0, lens[s]) for s in range(len(lens))])
                     for i in (0, 1))
    if case["op"] == "store":
        # codes are binary32 steps by definition (a code at a half goes where its product
        # rounds); what they stand for follows in 64 bits
        if case["seqs"] * case["rows"] > 1 << 20:
            return None
        outs = ([], [])
        for i, x in enumerate((st["k"], st["v"])):
            at = 0
            for s in range(len(lens)):
                if not rows[s]:
                    continue
                x_s = x[at:at + rows[s]].float()
                at += rows[s]
                lo = lens[s] - rows[s]
                for b in range(lo // page, -(-lens[s] // page)):
                    a, z = max(lo, b * page), min(lens[s], (b + 1) * page)
                    part = x_s[a - lo:z - lo]
                    scale = part.abs().amax((0, 2)).div(torch.full((h,), 127.0, device=x.device))
                    if a > b * page:
                        p = int(table[s, b])
                        was, kept = st["plain_scales"][p, :, i], st["codes"][i][p, :, :a - b * page]
                        grown = scale > was
                        scale = torch.where(grown, scale, was)
                        less = torch.where(grown, was / scale, torch.ones_like(was))
                        kept = torch.round(kept.float() * less[:, None, None]).to(f64)
                        outs[i].append((kept * scale.to(f64)[:, None, None]).transpose(0, 1))
                    inv = torch.where(scale > 0, scale.reciprocal(), 0.0)[:, None]
                    q = torch.round(part * inv).clamp(-127, 127).to(f64)
                    outs[i].append(q * scale.to(f64)[:, None])
        return torch.cat(outs[0]), torch.cat(outs[1])
    group, q, outs, lses = case["q_heads"] // h, st["q"].to(f64), [], []
    at = 0
    for s in range(len(lens)):
        k, v = (tokens(i, s, 0, lens[s]) for i in (0, 1))
        for r in range(0, rows[s], 512):
            m = min(512, rows[s] - r)
            x = q[at + r:at + r + m].view(m, h, group, dim).permute(1, 2, 0, 3).reshape(h, -1, dim)
            score = torch.matmul(x, k.permute(1, 2, 0).contiguous()) / math.sqrt(dim)
            p = lens[s] - rows[s] + r + torch.arange(m, device=x.device)
            j = torch.arange(lens[s], device=x.device)
            hidden = j[None] > p[:, None]
            if case["window"]:
                hidden |= j[None] <= p[:, None] - case["window"]
            score = score.view(h, group, m, -1).masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(score, 3)
            weight = torch.exp(score - lse[..., None]).view(h, group * m, -1)
            o = torch.matmul(weight, v.transpose(0, 1).contiguous()).view(h, group, m, dim)
            outs.append(o.permute(2, 0, 1, 3).reshape(m, -1, dim))
            lses.append(lse.permute(2, 0, 1).reshape(m, -1))
        at += rows[s]
    return torch.cat(outs), torch.cat(lses)


# ------------------------------------------------------------------- work --

def work(case):
    h, dim = case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        values = case["tokens"] * (case["q_heads"] + h) * dim
        size = {"bf16": 2, "f32": 4}
        return dict(bytes=values * (size[case["dtype"]] + size[case["out"]]) +
                    4 * case["tokens"] * (case["rot"] + 1) + 8 * dim, flops=10 * values)
    past, lens, rows = _lengths(case)
    each = 2 * h * dim                                     # keys and values of a token
    if case["op"] == "read":
        return dict(bytes=sum(lens) * each * (1 + (2 if case["out"] == "bf16" else 4)),
                    flops=sum(lens) * each)
    if case["op"] == "store":
        held = sum(p % case["page"] + n for p, n in zip(past, rows) if n)
        new = sum(rows)
        return dict(bytes=new * each * ((2 if case["dtype"] == "bf16" else 4) + 1) +
                    held * each * (1 + 4), flops=4 * new * each + held * each)
    pairs, used = 0, 0
    for p, n, length in zip(past, rows, lens):
        w = case["window"] or length
        first = max(0, p - w + 1)
        used += length - first if n else 0
        # rows see p + 1, p + 2, ... tokens, at most w
        grow = min(n, max(0, w - p))
        pairs += grow * p + grow * (grow + 1) // 2 + (n - grow) * w
    hq = case["q_heads"]
    return dict(bytes=used * each + sum(rows) * hq * (4 * dim + 4), flops=4 * dim * hq * pairs)

"""Plain models of the paged 8-bit cache and of attention over it, for the tests: the cache's
byte layout written out index by index, its binary32 quantization in numpy, attention in 64
bits with the error that the kernel's roundings can add up to."""
import numpy as np
import torch


def key_offset(token, d, dim):
    """Byte of element d of a token in the keys of a page."""
    c, r = d // 64, token % 16
    tile = token // 16 * 16 * dim
    if dim - 64 * c >= 64:
        return tile + 1024 * c + (16 * (d % 64 // 16) + r) * 16 + d % 16
    return tile + 1024 * c + (16 * (d % 64 // 8) + r) * 8 + d % 8


def value_offset(token, d, dim):
    c, r = d // 64, token % 16
    record = 16 if dim - 64 * c >= 64 else 8
    return (token // 16 * 16 * dim + 1024 * c + (16 * (r // 4) + d % 16) * record +
            d % 64 // 16 * 4 + r % 4)


def offsets(page, dim):
    """(keys, values): int64 [page, dim], the byte of each token's element."""
    t, d = np.meshgrid(np.arange(page), np.arange(dim), indexing="ij")
    k = np.vectorize(lambda a, b: key_offset(a, b, dim))(t, d)
    v = np.vectorize(lambda a, b: value_offset(a, b, dim))(t, d)
    return k, v


def pack(codes):
    """Codes int8 [2, pages, heads, page, dim] -> kv uint8 [pages, heads, 2, page, dim]."""
    _, pages, heads, page, dim = codes.shape
    kv = np.zeros((pages, heads, 2, page * dim), np.uint8)
    for i, at in enumerate(offsets(page, dim)):
        kv[:, :, i, at.reshape(-1)] = (codes[i].astype(np.int16) + 128).astype(np.uint8) \
            .reshape(pages, heads, -1)
    return kv.reshape(pages, heads, 2, page, dim)


def unpack(kv):
    pages, heads, _, page, dim = kv.shape
    flat = kv.reshape(pages, heads, 2, page * dim)
    return np.stack([(flat[:, :, i, at.reshape(-1)].astype(np.int16) - 128).astype(np.int8)
                     .reshape(pages, heads, page, dim)
                     for i, at in enumerate(offsets(page, dim))])


F = np.float32


def write(codes, scales, table, lens, starts, x):
    """x = (k, v) float32 [rows, heads, dim] into codes int8 [2, pages, heads, page, dim] and
    scales float32 [pages, heads, 2], in place, each step rounded to binary32."""
    page, pages = codes.shape[3], codes.shape[1]
    for s, length in enumerate(lens):
        n = starts[s + 1] - starts[s]
        lo = length - n
        for b in range(max(lo, 0) // page, -(-length // page) if n > 0 else 0):
            a, z = max(lo, b * page, 0), min(length, (b + 1) * page)
            if z <= a or b >= table.shape[1] or not 0 <= table[s, b] < pages:
                continue
            p = table[s, b]
            rows = slice(starts[s] + a - lo, starts[s] + z - lo)
            for i in range(2):
                new = x[i][rows].transpose(1, 0, 2)               # heads, tokens, dim
                with np.errstate(all="ignore"):
                    scale = np.abs(new).max((1, 2)).astype(F) / F(127)
                    old = a - b * page
                    if old:
                        was = scales[p, :, i].copy()
                        grown = scale > was
                        ratio = np.where(grown, was / np.where(grown, scale, F(1)), F(1)).astype(F)
                        scale = np.where(grown, scale, was)
                        c = np.rint(codes[i, p, :, :old].astype(F) * ratio[:, None, None])
                        codes[i, p, :, :old] = np.clip(c, -127, 127).astype(np.int8)
                    inv = np.where(scale > 0, F(1) / np.where(scale > 0, scale, F(1)), F(0))
                    q = new * inv.astype(F)[:, None, None]
                    q = np.where(np.isnan(q), F(0), np.clip(np.rint(q), -127, 127))
                codes[i, p, :, a - b * page:z - b * page] = q.astype(np.int8)
                scales[p, :, i] = scale


def read(codes, scales, table, lens, starts, rows, fill=np.nan):
    """(k, v) float32 [rows, heads, dim] of the last tokens; `fill` in rows of no token."""
    _, pages, heads, page, dim = codes.shape
    out = np.full((2, rows, heads, dim), fill, F)
    for s, length in enumerate(lens):
        n = starts[s + 1] - starts[s]
        for i in range(n):
            at = length - n + i
            if at < 0:
                continue
            b = at // page
            p = table[s, b] if b < table.shape[1] else -1
            if not 0 <= p < pages:
                out[:, starts[s] + i] = 0
                continue
            out[:, starts[s] + i] = codes[:, p, :, at % page].astype(F) * scales[p].T[:, :, None]
    return out


def attention(q, codes, scales, table, lens, starts, causal=True, window=0, scale=None,
              max_rows=None):
    """In 64 bits on q's device: (out, lse, err_out, err_lse), rows of no token NaN.

    q bfloat16 [rows, q_heads, dim], codes int8 [2, pages, heads, page, dim] and scales on the
    device too.  err_*: what the kernel's steps may be off by, from these bounds (u = 2^-24 a
    rounding of binary32, doubled for the matrix cores' sums, whose rounding is not specified):
      score   a sum of dim exact products and two more roundings, then the exponent's sum
              with log2 of the page's scale and the maximum:
              ds = 2 u (dim + 4) scale sum |q k| + 4 u (|s| + |lse| + 128)
      weight  exp2 adds 2^-22; p is rounded to 11 bits (2^-11), or where it is below 2^-14 of
              the unit to 2^-25 of that (times 127, a token: the unit is at most 1 / 1 of the
              largest p, so each token adds 2^-25 * 127 times the largest weight times scale)
      out     twice ds (numerator and denominator), sums over tokens of 2 u each,
              times A = sum w |v|; the output's rounding is left to the caller
    """
    rows, hq, dim = q.shape
    _, pages, heads, page, _ = codes.shape
    group = hq // heads
    if scale is None:
        scale = dim ** -0.5
    dev, f8 = q.device, torch.float64
    out = torch.full((rows, hq, dim), float("nan"), dtype=f8, device=dev)
    lse = torch.full((rows, hq), float("nan"), dtype=f8, device=dev)
    eo, el = out.clone(), lse.clone()
    u = 2.0 ** -24
    for s, length in enumerate(lens):
        n = starts[s + 1] - starts[s]
        m = min(n, max_rows) if max_rows else n
        if m <= 0:
            continue
        length = max(length, 0)
        at = torch.arange(length, device=dev)
        blocks = torch.as_tensor(table[s], device=dev).long()
        block = torch.cat([blocks, torch.full((length // page + 1,), -1, device=dev)])[at // page]
        have = (block >= 0) & (block < pages)
        block = torch.where(have, block, 0)
        p = length - n + torch.arange(m, device=dev)
        see = have[None].expand(m, -1).clone()
        if causal:
            see &= at[None] <= p[:, None]
        if window:
            see &= at[None] > p[:, None] - window
        if pages:
            kv = codes[:, block, :, at % page].to(f8).permute(1, 2, 0, 3)    # 2, heads, tokens, dim
            # what no row sees may hold anything
            sc = torch.where(see.any(0)[:, None, None], scales[block].to(f8), 0.0).permute(2, 1, 0)
            kv = kv * sc[..., None]
        else:
            kv = torch.zeros((2, heads, length, dim), dtype=f8, device=dev)
            sc = torch.zeros((2, heads, length), dtype=f8, device=dev)
        x = q[starts[s]:starts[s] + m].to(f8).view(m, heads, group, dim).permute(1, 2, 0, 3)
        x = x.reshape(heads, group * m, dim)
        score = torch.matmul(x, kv[0].transpose(1, 2)) * scale
        mass = torch.matmul(x.abs(), kv[0].abs().transpose(1, 2)) * abs(scale)
        see = see[None, None].expand(heads, group, m, length).reshape(heads, group * m, length)
        score = score.masked_fill(~see, float("-inf"))
        l = torch.logsumexp(score, 2) if length else \
            torch.full((heads, group * m), float("-inf"), dtype=f8, device=dev)
        some = l > float("-inf")
        w = torch.exp(score - torch.where(some, l, 0.0)[..., None])
        o = torch.matmul(w, kv[1])
        a = torch.matmul(w, kv[1].abs())
        if length:
            worst = torch.where(see, mass, 0.0).amax(2)
            ds = 2 * u * (dim + 4) * worst + 4 * u * (2 * l.abs().nan_to_num(0, 0, 0) + 128)
            ds = ds + 4 * u * worst
            unit = (w * sc[1][:, None, :]).amax(2)
        else:
            ds, unit = torch.zeros_like(l), torch.zeros_like(l)
        rel = 2 * ds + 2.0 ** -11 + 2.0 ** -21 + 2 * u * (length + 64)
        bound = rel[..., None] * a + (length * 2.0 ** -25 * 127 * unit)[..., None]
        bl = ds + 2.0 ** -21 + 2 * u * (length + 64) + 2 * u * l.abs().nan_to_num(0, 0, 0)

        def back(t):
            return t.view(heads, group, m, -1).permute(2, 0, 1, 3).reshape(m, hq, -1)

        r = slice(starts[s], starts[s] + m)
        out[r], eo[r] = back(o), back(bound)
        lse[r], el[r] = back(l)[..., 0], back(bl)[..., 0]
    return out, lse, eo, el


def make_table(lens, page, pages, rng, blocks=None):
    """Block tables int32 [seqs, blocks] over pages in random order, -1 where none is needed."""
    need = [-(-max(x, 0) // page) for x in lens]
    order = rng.permutation(pages)[:sum(need)]
    assert len(order) == sum(need)
    table = np.full((len(lens), blocks or max(need + [1])), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table


def starts_of(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)

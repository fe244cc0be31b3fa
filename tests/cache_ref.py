"""Quantized matrices and paged caches in binary64: what the codes stand for, where a
batch's tokens lie, attention over them."""
import torch

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def e4m3_values(dev):
    c = torch.arange(256, dtype=torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.double() - 10)) * (1 - 2.0 * (c >> 7))
    v[(c & 127) == 127] = float("nan")
    return v.to(dev)


def values(codes, scales, fmt, s2=None):
    """Codes [..., bytes] and scales [..., blocks] -> binary64 [..., n]; s2: of each row."""
    dev = codes.device
    e4m3 = e4m3_values(dev)
    if fmt == "mxfp8":
        v = e4m3[codes.long()]
    else:
        b = codes.long()
        v = E2M1.to(dev)[torch.stack((b & 15, b >> 4), -1).flatten(-2)]
    if fmt == "nvfp4":
        d = e4m3[scales.long()] * s2.double()[..., None]
    else:
        d = torch.ldexp(torch.ones_like(scales, dtype=torch.float64), scales.int() - 127)
    return v * d.repeat_interleave(v.shape[-1] // d.shape[-1], -1)


def places(cu, lens, table, page_tokens, pages):
    """Of each row that has one: (row, sequence, position, page, token of the page)."""
    cu, lens, table = cu.tolist(), lens.tolist(), table.tolist()
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            pos = lens[b] - n + i
            if pos < 0:
                continue
            at = pos // page_tokens
            page = table[b][at] if at < len(table[b]) else -1
            if 0 <= page < pages:
                yield cu[b] + i, b, pos, page, pos % page_tokens


def sequence_values(cache, b, lens, table):
    """Keys and values of sequence b, binary64 [len, kv_heads, dim] each."""
    n = max(int(lens[b]), 0)
    t = torch.arange(n, device=cache.device)
    page, tok = table[b].long()[t // cache.page_tokens], t % cache.page_tokens
    out = []
    for codes, scales, s2 in ((cache.k_codes, cache.k_scales, cache.k_s2), (cache.v_codes, cache.v_scales, cache.v_s2)):
        s = None if s2 is None else s2[None].expand(n, -1)
        out.append(values(codes[page, :, tok], scales[page, :, tok], cache.fmt, s))
    return out


def attention(cache, q, cu, lens, table, scale):
    """(o, lse, weight, spread): weight [T, heads, dim] = sum_j p_j |v_j|, spread [T, heads] =
    |scale| max_j sum_d |q_d k_jd|.  Rows of no sequence: zeros."""
    T, heads, dim = q.shape
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=q.device)  # noqa: E731
    o, lse, weight, spread = z(T, heads, dim), z(T, heads), z(T, heads, dim), z(T, heads)
    for b in range(len(lens)):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        if r1 <= r0:
            continue
        k, v = sequence_values(cache, b, lens, table)
        g = heads // cache.kv_heads
        k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
        x = q[r0:r1].double()
        pos = int(lens[b]) - (r1 - r0) + torch.arange(r1 - r0, device=q.device)
        s = scale * torch.einsum("ihd,jhd->ihj", x, k)
        seen = torch.arange(k.shape[0], device=q.device)[None] <= pos[:, None]
        s = s.masked_fill(~seen[:, None], float("-inf"))
        l = torch.logsumexp(s, -1) if k.shape[0] else torch.full((r1 - r0, heads), float("-inf"), device=q.device).double()
        p = torch.exp(s - torch.where(l.isinf(), 0.0, l)[..., None])
        o[r0:r1], lse[r0:r1] = torch.einsum("ihj,jhd->ihd", p, v), l
        weight[r0:r1] = torch.einsum("ihj,jhd->ihd", p, v.abs())
        if k.shape[0]:
            spread[r0:r1] = abs(scale) * torch.einsum("ihd,jhd->ihj", x.abs(), k.abs()).amax(-1)
    return o, lse, weight, spread

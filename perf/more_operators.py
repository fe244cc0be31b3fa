"""Workloads of the operators that run the attention half of a converted layer: products of a few tokens with 4-bit and 8-bit
weights, a key/value cache that is quantized as it is written and read back, and attention of new tokens over that cache.

`listed()` names the workloads, `draw()` gives more of the same ranges, `prepare()` makes a case's data on the GPU, `run()`
passes once through the operator (in elementary torch operations, or through the library where `own` is true), `exact()`
states the result in binary64 and `work()` counts the bytes and operations that cannot be avoided.

Weights have the sizes of the converter's workloads (hidden 2048, the shared expert's 2560 x 2048 and 2048 x 1280 matrices) and
those of an output head. A cache holds its tokens in pages, [pages, kv_heads, page_tokens, head_dim] codes with one scale per 32
(MXFP8) or 16 (NVFP4) values of a head, keys and values apart. A batch of sequences is described by `cu` (first row of
each sequence's new tokens, and the end), `lens` (tokens of each sequence in the cache, the new ones among them) and `table`
(the pages of each sequence): row i of a sequence with n rows stands for its position len - n + i.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
OUTLIERS = (101, 717, 1333, 1949)   # channels of a token tile that are 30 times as large


def listed():
    return [
        # shared expert's gate and up for one token, 4-bit: latency
        {"name": "linear nvfp4 1x2560x2048", "op": "linear", "t": 1, "n": 2560, "k": 2048, "fmt": "nvfp4", "out": "bf16"},
        # its down projection for a small decoding batch
        {"name": "linear mxfp8 16x2048x1280", "op": "linear", "t": 16, "n": 2048, "k": 1280, "fmt": "mxfp8", "out": "bf16"},
        # an output head for one token, logits in fp32: the read of the weights
        {"name": "linear nvfp4 1x65536x2048 f32", "op": "linear", "t": 1, "n": 65536, "k": 2048, "fmt": "nvfp4", "out": "f32"},
        # the same for a decoding batch, a ragged number of tokens and of outputs
        {"name": "linear mxfp4 27x50001x2048", "op": "linear", "t": 27, "n": 50001, "k": 2048, "fmt": "mxfp4", "out": "bf16"},
        # one new token of each of 16 sequences, written and seen again: latency; a padding row
        {"name": "store mxfp8 16 tokens", "op": "store", "seqs": 16, "new": 1, "ctx": 2000, "ragged": 3, "pad": 1, "kv": 2,
         "dim": 128, "page": 64, "fmt": "mxfp8", "mode": "rtn"},
        # a prefill of 17000 tokens in sequences of different lengths: bandwidth
        {"name": "store nvfp4 17000 tokens", "op": "store", "seqs": 8, "new": 4096, "ctx": 8192, "ragged": 11, "pad": 0,
         "kv": 8, "dim": 128, "page": 64, "fmt": "nvfp4", "mode": "four_six"},
        # a cache handed over: all tokens of 24 sequences back in bf16
        {"name": "load mxfp8 24 sequences", "op": "load", "seqs": 24, "ctx": 8192, "ragged": 5, "kv": 4, "dim": 128,
         "page": 16, "fmt": "mxfp8"},
        # one short sequence in 4 bits
        {"name": "load nvfp4 777 tokens", "op": "load", "seqs": 1, "ctx": 777, "ragged": 0, "kv": 2, "dim": 256, "page": 32,
         "fmt": "nvfp4"},
        # a decoding step of one sequence: latency, the read of its cache spread over the card
        {"name": "attention mxfp8 1x1 over 5000", "op": "attention", "seqs": 1, "new": 1, "ctx": 5000, "ragged": 0, "pad": 0,
         "kv": 2, "group": 8, "dim": 128, "page": 64, "fmt": "mxfp8"},
        # a decoding step of a large batch of sequences of up to 32768 tokens: the read of the caches
        {"name": "attention mxfp8 64x1 over 32768", "op": "attention", "seqs": 64, "new": 1, "ctx": 32768, "ragged": 7,
         "pad": 2, "kv": 2, "group": 8, "dim": 128, "page": 64, "fmt": "mxfp8"},
        # several guessed tokens a sequence, 4-bit cache, wide heads
        {"name": "attention nvfp4 12x4 over 16384", "op": "attention", "seqs": 12, "new": 4, "ctx": 16384, "ragged": 9,
         "pad": 0, "kv": 2, "group": 8, "dim": 256, "page": 32, "fmt": "nvfp4"},
        # a chunk of a long prompt: the products
        {"name": "attention mxfp8 1x4096 over 20480", "op": "attention", "seqs": 1, "new": 4096, "ctx": 20480, "ragged": 0,
         "pad": 0, "kv": 4, "group": 8, "dim": 128, "page": 64, "fmt": "mxfp8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "store", "load", "attention", "attention", "attention"))
    if op == "linear":
        t, k = _log(rng, 1, 64), 32 * _log(rng, 1, 256)
        n = _log(rng, 1, min(65536, 65536 * 2048 // k, 27 * 65536 * 2048 // (t * k)))
        return {"op": op, "t": t, "n": n, "k": k, "fmt": rng.choice(("nvfp4", "nvfp4", "mxfp4", "mxfp8")),
                "out": rng.choice(("bf16", "bf16", "f32"))}
    c = {"op": op, "seqs": _log(rng, 1, 64), "ragged": rng.randint(1, 10 ** 6), "kv": rng.choice((1, 2, 4, 8)),
         "dim": rng.choice((64, 128, 128, 256)), "page": rng.choice((16, 32, 64, 128)), "fmt": rng.choice(("mxfp8", "nvfp4"))}
    width = c["seqs"] * c["kv"] * c["dim"]
    if op == "load":
        return dict(c, ctx=_log(rng, 1, min(32768, 24 * 8192 * 4 * 128 // width)))
    if op == "store":
        new = _log(rng, 1, min(4096, 8 * 4096 * 8 * 128 // width))
        return dict(c, new=new, ctx=new + _log(rng, 1, 4096), pad=rng.choice((0, 0, 3)),
                    mode=rng.choice(("rtn", "four_six")) if c["fmt"] == "nvfp4" else "rtn")
    group = rng.randint(1, 16)
    ctx = _log(rng, 1, min(65536, 64 * 32768 * 2 * 128 // width))
    pairs = 4096 * 20480 * 32 * 128 // (width * group * ctx)        # new tokens a sequence that the largest case allows
    new = rng.choice((1, 1, rng.randint(2, 8), _log(rng, 16, 4096)))
    return dict(c, group=group, ctx=ctx, new=max(1, min(new, ctx, pairs)), pad=rng.choice((0, 0, 3)))


def _lens(case):
    """New tokens and tokens in the cache of each sequence."""
    b, ctx, new = case["seqs"], case["ctx"], case.get("new", case["ctx"])
    if not case["ragged"]:
        return [new] * b, [ctx] * b
    r = random.Random(case["ragged"])
    lens = [ctx] + [_log(r, max(1, ctx // 16), ctx) for _ in range(b - 1)]
    if case["op"] == "load":
        return list(lens), lens
    news = [min(n, new if new <= 8 else r.randint(max(1, new // 2), new)) for n in lens]
    if b > 3:
        news[2] = 0     # a sequence that sits this step out
    return news, lens


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def _rows(x, fmt, s2, mode="rtn"):
    """Values, codes (a byte each) and block scales (bytes) of the last dimension of x (bf16 values), s2: a global scale for
    each row, where the format has one."""
    b = x.float().unflatten(-1, (-1, BLOCK[fmt]))
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        codes, scale, d = _nvfp4(b, amax, s2[..., None, None], 6.0)
        if mode == "four_six":
            c4, s4, d4 = _nvfp4(b, amax, s2[..., None, None], 4.0)
            less = _excess(b, c4, s4, s2) < _excess(b, codes, scale, s2)
            codes, scale, d = (torch.where(less, u, v) for u, v in ((c4, codes), (s4.view(torch.uint8), scale.view(torch.uint8)), (d4, d)))
        return (_e2m1(codes) * scale.view(torch.float8_e4m3fn).float() * s2[..., None, None]).flatten(-2), codes.flatten(-2), scale.view(torch.uint8)[..., 0]
    m, e = torch.frexp(amax / (448.0 if fmt == "mxfp8" else 6.0))       # amax <= top 2^e, the smallest such e
    e = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
    y = torch.ldexp(b, -e)
    if fmt == "mxfp8":
        codes = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        v, codes = codes.float(), codes.view(torch.uint8)
    else:
        codes = _to_e2m1(y)
        v = _e2m1(codes)
    return torch.ldexp(v, e).flatten(-2), codes.flatten(-2), torch.where(amax > 0, e + 127, 0).to(torch.uint8)[..., 0]


def _nvfp4(b, amax, s2, top):
    scale = torch.nan_to_num(amax / (top * s2), 0.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = scale.float() * s2
    return torch.where(d > 0, _to_e2m1(b / torch.where(d > 0, d, 1.0)), 0), scale, d


def _excess(b, codes, scale, s2):
    """Squared error of a block less its sum of squares, over s2: the 4/6 rule takes the smaller one."""
    q, d = _e2m1(codes).double(), scale.double()
    return (d * (d * s2[..., None, None].double() * q.square().sum(-1, keepdim=True) - 2.0 * (q * b.double()).sum(-1, keepdim=True)))


def _to_e2m1(y):
    """E2M1 codes, ties to the even one."""
    a = y.abs()
    n = sum((a > t).to(torch.uint8) if i % 2 == 0 else (a >= t).to(torch.uint8)
            for i, t in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    return n + 8 * torch.signbit(y).to(torch.uint8)


def _e2m1(codes):
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    return lut[codes.int()]


def _packed(codes, fmt):
    return codes if fmt == "mxfp8" else codes[..., 0::2] | (codes[..., 1::2] << 4)


def _decode(codes, scales, fmt, s2):
    """fp32 values of packed codes and block scales; s2: a global scale for each row."""
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        v = _e2m1(torch.stack((codes & 15, codes >> 4), -1).flatten(-2))
    if fmt == "nvfp4":
        d = scales.view(torch.float8_e4m3fn).float() * s2[..., None]
    else:
        d = torch.where(scales > 0, (scales.int() << 23).view(torch.float32), 2.0 ** -127)
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * d[..., None]).flatten(-2)


def _pool(shape, fmt, s2, spread, g):
    """Codes and scales of `shape` values, [pages, kv_heads, page_tokens, head_dim]: N(0, 1) times a factor of the token, and
    four channels `spread` times as large. 2^24 values at a time."""
    codes, scales = [], []
    step = max(1, (1 << 24) // (shape[1] * shape[2] * shape[3]))
    for p in range(0, shape[0], step):
        n = min(step, shape[0] - p)
        x = _randn((n,) + shape[1:], g) * torch.exp(0.3 * _randn((n,) + shape[1:3] + (1,), g))
        x[..., ::shape[3] // 4] *= spread
        _, c, s = _rows(x.to(torch.bfloat16), fmt, None if s2 is None else s2[None, :, None].expand(x.shape[:-1]))
        codes.append(_packed(c, fmt))
        scales.append(s)
    return torch.cat(codes), torch.cat(scales)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "linear":
        t, n, k, fmt = case["t"], case["n"], case["k"], case["fmt"]
        x = _randn((t, k), g)
        for c in OUTLIERS:
            if c < k:
                x[:, c] *= 30.0
        s["x"] = x.to(torch.bfloat16)
        w = (_randn((n, k), g) * 0.02).to(torch.bfloat16)
        s["s2"] = (w.abs().amax().float() / 2688.0).view(1) if fmt == "nvfp4" else None
        codes, scales = [], []
        step = max(1, (1 << 25) // k)
        for r in range(0, n, step):
            _, c, sc = _rows(w[r:r + step], fmt, None if s["s2"] is None else s["s2"].expand(len(w[r:r + step])))
            codes.append(_packed(c, fmt))
            scales.append(sc)
        s["codes"], s["scales"] = torch.cat(codes), torch.cat(scales)
        s["y"] = torch.empty((t, n), dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device=DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return s
    news, lens = _lens(case)
    kv, dim, page, fmt = case["kv"], case["dim"], case["page"], case["fmt"]
    rows = sum(news) + case.get("pad", 0)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + 3, generator=g, device=DEV).to(torch.int32)
    s["table"] = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        s["table"][b, :n] = order[at:at + n]
        at += n
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["max_new"], s["max_len"] = max(news), max(lens)
    s["k_s2"] = s["v_s2"] = None
    if fmt == "nvfp4":      # what a calibration gave for each head
        s["k_s2"] = torch.exp(0.1 * _randn(kv, g)) * (30.0 / 2688.0)
        s["v_s2"] = torch.exp(0.1 * _randn(kv, g)) * (9.0 / 2688.0)
    shape = (sum(need) + 3, kv, page, dim)
    s["k_codes"], s["k_scales"] = _pool(shape, fmt, s["k_s2"], 6.0, g)
    s["v_codes"], s["v_scales"] = _pool(shape, fmt, s["v_s2"], 1.0, g)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if case["op"] == "attention":
        heads = kv * case["group"]
        s["q"] = _randn((rows, heads, dim), g).to(torch.bfloat16)
        s["o"] = torch.zeros((rows, heads, dim), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((rows, heads), dtype=torch.float32, device=DEV)
        return s
    if case["op"] == "store":
        # keys and values as a projection leaves them: columns of one tensor
        s["kv_new"] = (_randn((rows, 2, kv, dim), g) * torch.exp(0.3 * _randn((rows, 2, kv, 1), g))).to(torch.bfloat16)
    s["k"] = torch.zeros((rows, kv, dim), dtype=torch.bfloat16, device=DEV)
    s["v"] = torch.zeros((rows, kv, dim), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------- plain forms --
def _places(s):
    """Of the rows that belong to a sequence: their numbers, and their token's place, page and row in the page."""
    rows = torch.arange(s["k"].shape[0], device=DEV)
    rows = rows[:int(sum(_lens(s)[0]))]
    b = torch.searchsorted(s["cu"], rows.to(torch.int32), right=True) - 1
    pos = s["lens"][b] - (s["cu"][b + 1] - s["cu"][b]) + rows - s["cu"][b]
    return rows, s["table"][b, pos // s["page"]].long(), pos % s["page"]


def _plain_cache(s):
    rows, page, at = _places(s)
    out = {}
    for i, name in enumerate("kv"):
        codes, scales, s2 = s[name + "_codes"], s[name + "_scales"], s[name + "_s2"]
        per_row = None if s2 is None else s2[None].expand(len(rows), -1)
        if s["op"] == "store":
            _, c, sc = _rows(s["kv_new"][rows, i], s["fmt"], per_row, s["mode"])
            codes[page, :, at] = _packed(c, s["fmt"])
            scales[page, :, at] = sc
        s[name][rows] = _decode(codes[page, :, at], scales[page, :, at], s["fmt"], per_row).to(torch.bfloat16)
        out[name] = s[name]
    return out


def _cached(s, name, at):
    """fp32 keys or values of the positions `at` (one row of them for all sequences), [sequence, kv_heads, position, dim]."""
    page = s["table"].clamp(min=0)[:, at // s["page"]].long()
    row = (at % s["page"]).expand_as(page)
    codes, scales, s2 = s[name + "_codes"], s[name + "_scales"], s[name + "_s2"]
    return _decode(codes[page, :, row], scales[page, :, row], s["fmt"], None if s2 is None else s2.expand(page.shape + (-1,))).transpose(1, 2)


def _plain_attention(s):
    q, kv, g, d, m = s["q"], s["kv"], s["group"], s["dim"], s["max_new"]
    rows = torch.arange(int(sum(_lens(s)[0])), device=DEV)
    b = torch.searchsorted(s["cu"], rows.to(torch.int32), right=True) - 1
    i = rows - s["cu"][b]
    n = s["cu"][1:] - s["cu"][:-1]
    at = torch.arange(s["max_len"], device=DEV)
    qp = torch.zeros((len(n), m, kv, g, d), device=DEV)
    qp[b, i] = q[rows].float().view(-1, kv, g, d)
    sc = torch.matmul(qp.permute(0, 2, 3, 1, 4).reshape(len(n), kv, g * m, d), _cached(s, "k", at).transpose(2, 3))
    sc = sc.view(len(n), kv, g, m, -1).mul_(1.0 / math.sqrt(d))
    pos = (s["lens"] - n)[:, None] + torch.arange(m, device=DEV)
    sc.masked_fill_((at > pos[..., None])[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _cached(s, "v", at).masked_fill((at >= s["lens"][:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.view(len(n), kv, g * m, -1), v).view(len(n), kv, g, m, d) / total.clamp(min=1e-30)
    s["o"][rows] = o.permute(0, 3, 1, 2, 4)[b, i].reshape(-1, kv * g, d).to(torch.bfloat16)
    s["lse"][rows] = (top + total.log())[..., 0].permute(0, 3, 1, 2)[b, i].reshape(-1, kv * g)
    return {"o": s["o"], "lse": s["lse"]}


def _own_cache(s):
    from mxfp_block_scaled_b200 import mxq
    if "cache" not in s:   # a program's handle of its cache
        s["cache"] = mxq.Cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["fmt"], s["k_s2"], s["v_s2"])
    return mxq, s["cache"]


def run(state):
    s = state
    if own:
        if s["op"] == "linear":
            from mxfp_block_scaled_b200 import mxq
            if "workspace" not in s:   # kept by the caller from call to call
                s["workspace"] = mxq.linear_workspace(s["t"], s["k"], s["x"].device)
            mxq.mxq_linear(s["x"], s["t"], s["k"], s["fmt"], s["codes"], s["scales"], s["s2"], s["n"], s["out"], s["y"], s["status"],
                           s["workspace"])
            return {"y": s["y"]}
        mxq, cache = _own_cache(s)
        batch, nb, width = (s["cu"], s["lens"], s["table"]), len(s["lens"]), s["table"].shape[1]
        if s["op"] == "attention":
            if "workspace" not in s:
                s["workspace"] = mxq.cache_attention_workspace(cache, len(s["q"]), s["q"].shape[1], nb, s["max_new"])
            mxq.mxq_cache_attention(cache, s["q"], s["q"].stride(0), len(s["q"]), s["q"].shape[1], *batch, nb, width, s["max_new"],
                                    1.0 / math.sqrt(s["dim"]), s["o"], s["lse"], s["status"], s["workspace"])
            return {"o": s["o"], "lse": s["lse"]}
        if s["op"] == "store":
            k, v = s["kv_new"][:, 0], s["kv_new"][:, 1]
            mxq.mxq_cache_write(cache, k, k.stride(0), v, v.stride(0), len(k), *batch, nb, width, s["mode"], s["status"])
        mxq.mxq_cache_read(cache, *batch, nb, width, len(s["k"]), s["k"], s["v"], s["status"])
        return {"k": s["k"], "v": s["v"]}
    if s["op"] == "linear":
        w = _decode(s["codes"], s["scales"], s["fmt"], None if s["s2"] is None else s["s2"].expand(s["n"]))
        return {"y": torch.matmul(s["x"].float(), w.t()).to(s["y"].dtype)}
    return _plain_attention(s) if s["op"] == "attention" else _plain_cache(s)


# -------------------------------------------------------------- definition --
def _e4m3_values():
    """The value of each E4M3 byte, from its fields."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(math.nan if c & 127 == 127 else -x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _values64(codes, scales, fmt, s2, e4m3):
    """A matrix [rows, cols] in binary64; s2: of each row."""
    if fmt == "mxfp8":
        v = e4m3[codes.long()]
    else:
        grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
        n = torch.stack((codes % 16, codes.div(16, rounding_mode="floor")), -1).reshape(codes.shape[0], -1).long()
        v = grid[n % 8] * (1 - 2 * (n // 8)).double()
    if fmt == "nvfp4":
        d = e4m3[scales.long()] * s2.double()[:, None]
    else:
        d = torch.ldexp(torch.ones_like(scales, dtype=torch.float64), scales.long() - 127)
    return v * d[:, torch.arange(v.shape[1], device=DEV) // (v.shape[1] // d.shape[1])]


def _nearest(x, grid):
    """The nearest of the ascending values `grid`, whose even places win ties; the sign is x's."""
    a = x.abs()
    hi = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)
    lo = hi - 1
    up = a - grid[lo], grid[hi] - a
    return torch.where((up[0] > up[1]) | ((up[0] == up[1]) & (hi % 2 == 0)), grid[hi], grid[lo]) * torch.sign(x)


def _stored64(x, fmt, s2, mode, e4m3):
    """What a cache holds of the rows x [rows, dim], in binary64; the quotients are rounded to fp32 as the format defines."""
    e4 = e4m3[:127]
    e2 = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    b = x.double().view(x.shape[0], -1, BLOCK[fmt])
    amax = b.abs().amax(2, keepdim=True)
    if fmt != "nvfp4":
        e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448.0))
        e = torch.where(448.0 * torch.exp2(e - 1) >= amax, e - 1, torch.where(448.0 * torch.exp2(e) < amax, e + 1, e)).clamp(-127, 127)
        return (_nearest(b * torch.exp2(-e), e4) * torch.exp2(e)).view(x.shape)
    s2 = s2.double()[:, None, None]
    best = worst = None
    for top in (6.0, 4.0) if mode == "four_six" else (6.0,):
        scale = _nearest((amax / (top * s2).float().double()).float().double(), e4)
        d = (scale * s2).float().double()
        v = _nearest((b / torch.where(d > 0, d, 1.0)).float().double() * (d > 0), e2) * scale * s2
        err = (v * v - 2.0 * v * b).sum(2, keepdim=True)
        best, worst = (v, err) if best is None else (torch.where(err < worst, v, best), torch.minimum(err, worst))
    return best.view(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    e4m3 = _e4m3_values()
    fmt = case["fmt"]
    if case["op"] == "linear":
        y, x = [], s["x"].double()
        for r in range(0, case["n"], 8192):
            w = _values64(s["codes"][r:r + 8192], s["scales"][r:r + 8192], fmt, None if fmt != "nvfp4" else s["s2"].expand(len(s["codes"][r:r + 8192])), e4m3)
            y.append(x @ w.t())
        return {"y": torch.cat(y, 1)}
    news, lens = _lens(case)
    kv, page, dim = case["kv"], case["page"], case["dim"]
    rows = sum(news) + case.get("pad", 0)

    def held(name, b, h, n):
        """Tokens 0 .. n - 1 of sequence b and head h."""
        p = s["table"][b, :-(-n // page)].long()
        codes, scales = s[name + "_codes"][p, h].flatten(0, 1)[:n], s[name + "_scales"][p, h].flatten(0, 1)[:n]
        return _values64(codes, scales, fmt, s["k_s2" if name == "k" else "v_s2"][h].expand(n) if fmt == "nvfp4" else None, e4m3)

    if case["op"] != "attention":
        out = {name: torch.zeros((rows, kv, dim), dtype=torch.float64, device=DEV) for name in "kv"}
        for i, name in enumerate("kv"):
            for h in range(kv):
                if case["op"] == "store":
                    n = sum(news)
                    s2 = s[name + "_s2"][h].expand(n) if fmt == "nvfp4" else None
                    out[name][:n, h] = _stored64(s["kv_new"][:n, i, h], fmt, s2, case["mode"], e4m3)
                    continue
                at = 0
                for b, n in enumerate(lens):
                    out[name][at:at + n, h] = held(name, b, h, n)
                    at += n
        return out
    g = case["group"]
    o = torch.zeros((rows, kv * g, dim), dtype=torch.float64, device=DEV)
    lse = torch.zeros((rows, kv * g), dtype=torch.float64, device=DEV)
    at = 0
    for b, (new, n) in enumerate(zip(news, lens)):
        if not new:
            continue
        later = torch.arange(n, device=DEV)[None] > (torch.arange(new, device=DEV) + n - new)[:, None]
        for h in range(kv):
            k, v = held("k", b, h, n), held("v", b, h, n)
            for j in range(h * g, h * g + g):
                z = (s["q"][at:at + new, j].double() @ k.t() / math.sqrt(dim)).masked_fill_(later, -math.inf)
                lse[at:at + new, j] = torch.logsumexp(z, 1)
                o[at:at + new, j] = torch.exp(z - lse[at:at + new, j, None]) @ v
        at += new
    return {"o": o, "lse": lse}


# -------------------------------------------------------------------- work --
def work(case):
    per = {"nvfp4": 0.5 + 1 / 16, "mxfp4": 0.5 + 1 / 32, "mxfp8": 1 + 1 / 32}[case["fmt"]]
    if case["op"] == "linear":
        t, n, k = case["t"], case["n"], case["k"]
        return {"bytes": n * k * per + 2 * t * k + t * n * (4 if case["out"] == "f32" else 2), "flops": 2 * t * n * k}
    news, lens = _lens(case)
    width = 2 * case["kv"] * case["dim"]        # of a token's keys and values
    if case["op"] == "load":
        return {"bytes": sum(lens) * width * (per + 2), "flops": sum(lens) * width}
    if case["op"] == "store":
        return {"bytes": sum(news) * width * (2 + per + 2), "flops": 3 * sum(news) * width}
    heads, d = case["kv"] * case["group"], case["dim"]
    seen = sum(n * new - new * (new - 1) // 2 for new, n in zip(news, lens))
    return {"bytes": sum(n for new, n in zip(news, lens) if new) * width * per + sum(news) * heads * (4 * d + 4),
            "flops": 4 * d * heads * seen}

"""Workloads of the operators that run a converted layer: the block-FP8 quantizer, the block-FP8 matrix product and the
mixture-of-experts layer for a few tokens.

`listed()` names the workloads, `draw()` gives more of the same ranges, `prepare()` makes a case's data on the GPU, `run()`
passes once through the operator (in elementary torch operations, or through the library where `own` is true), `exact()`
states the result in binary64 and `work()` counts the bytes and operations that cannot be avoided.

Sizes are those of the converter's workloads: hidden 2048, expert width 768, 512 routed experts of which ten serve a token,
the shared expert's 2560 x 2048 and 2048 x 1280 matrices, token tiles of 1 to 65536 tokens, the tiny layer of 8 experts,
and ragged sizes between them.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
OUTLIERS = (101, 717, 1333, 1949)   # channels of a token tile that are 30 times as large


def listed():
    return [
        # one token's hidden state before the shared expert: the quantizer's latency
        {"name": "quantize 1 token", "op": "quantize", "rows": 1, "cols": 2048, "brows": 1},
        # the largest token tile of the activation sweep: bandwidth
        {"name": "quantize 65536 tokens", "op": "quantize", "rows": 65536, "cols": 2048, "brows": 1},
        # weights: the gate_up slabs of the 64 experts that the streaming converter holds at a time
        {"name": "quantize 64 gate_up slabs", "op": "quantize", "rows": 98304, "cols": 2048, "brows": 128},
        # shared expert, gate and up of one token: latency and the weights' read
        {"name": "gemm 1x2560x2048", "op": "gemm", "m": 1, "n": 2560, "k": 2048, "out": "bf16"},
        # shared expert, down projection of a small decoding batch
        {"name": "gemm 16x2048x1280", "op": "gemm", "m": 16, "n": 2048, "k": 1280, "out": "bf16"},
        # ragged in every direction (a tensor-parallel slice, a last block of 16), fp32 result
        {"name": "gemm 300x1999x1552 f32", "op": "gemm", "m": 300, "n": 1999, "k": 1552, "out": "f32"},
        # shared expert, gate and up of a prefill chunk
        {"name": "gemm 4096x2560x2048", "op": "gemm", "m": 4096, "n": 2560, "k": 2048, "out": "bf16"},
        # the same over the largest token tile
        {"name": "gemm 65536x2560x2048", "op": "gemm", "m": 65536, "n": 2560, "k": 2048, "out": "bf16"},
        # the tiny layer of the tests in the retained layers' format, two of five rows of the batch without a token
        {"name": "moe fp8 tiny 5 tokens", "op": "moe", "tokens": 5, "topk": 4, "experts": 8, "hidden": 256, "inter": 128,
         "fmt": "fp8_block", "padded": 2},
        # full-size layer, one token: the decoding step
        {"name": "moe nvfp4 1 token", "op": "moe", "tokens": 1, "topk": 10, "experts": 512, "hidden": 2048, "inter": 768,
         "fmt": "nvfp4", "padded": 0},
        # full-size layer of the mixed-format model, a small decoding batch
        {"name": "moe mxfp4 16 tokens", "op": "moe", "tokens": 16, "topk": 10, "experts": 512, "hidden": 2048, "inter": 768,
         "fmt": "mxfp4", "padded": 0},
        # full-size layer, the largest decoding batch that still counts as a few tokens; three rows are padding
        {"name": "moe nvfp4 64 tokens", "op": "moe", "tokens": 64, "topk": 10, "experts": 512, "hidden": 2048, "inter": 768,
         "fmt": "nvfp4", "padded": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "moe", "moe"))
    if op == "quantize":
        cols = 16 * _log(rng, 1, 512)
        return {"op": op, "rows": _log(rng, 1, min(65536, 65536 * 2048 // cols)), "cols": cols,
                "brows": rng.choice((1, 128))}
    if op == "gemm":
        k, n = 16 * _log(rng, 1, 512), _log(rng, 1, 8192)
        return {"op": op, "m": _log(rng, 1, min(65536, 65536 * 2560 * 2048 // (n * k), 65536 * 2560 // n)), "n": n, "k": k,
                "out": rng.choice(("bf16", "bf16", "f32"))}
    hidden, inter = 128 * _log(rng, 1, 16), 128 * _log(rng, 1, 6)
    experts = _log(rng, 4, 512)
    topk = rng.randint(1, min(10, experts))
    tokens = _log(rng, 1, 64)
    return {"op": op, "tokens": tokens, "topk": topk, "experts": experts, "hidden": hidden, "inter": inter,
            "fmt": rng.choice(("nvfp4", "nvfp4", "mxfp4", "mxfp8", "fp8_block")),
            "padded": rng.choice((0, 0, tokens // 8))}


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _tokens(t, hidden, g):
    """A token tile: N(0, 1) with a few channels 30 times as large."""
    x = torch.randn((t, hidden), generator=g, device=DEV)
    for c in OUTLIERS:
        if c < hidden:
            x[:, c] *= 30.0
    return x.to(torch.bfloat16)


def _blocks(x, brows):
    """Largest magnitude of each brows x 128 block of a matrix, ragged edges included."""
    rows, cols = x.shape
    p = torch.nn.functional.pad(x.abs(), (0, -cols % 128, 0, -rows % brows))
    return p.view(p.shape[0] // brows, brows, p.shape[1] // 128, 128).amax((1, 3))


def _spread(s, brows, rows, cols):
    """A block's scale at each value of the block."""
    return s.repeat_interleave(brows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def _quantize(x, brows):
    """E4M3 codes (as float8) and the fp32 scale of each brows x 128 block."""
    x = x.float()
    s = _blocks(x, brows) / 448.0
    d = _spread(s, brows, *x.shape)
    y = torch.where(d > 0, x / d, torch.zeros_like(x)).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), s


def _experts(e, rows, cols, fmt, std, g):
    """Stacked expert weights in `fmt`, drawn and rounded 64 experts at a time: codes, scales, global scales."""
    codes, scales, s2s = [], [], []
    edges = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=DEV)
    for e0 in range(0, e, 64):
        n = min(64, e - e0)
        w = torch.randn((n, rows, cols), generator=g, device=DEV) * std[e0:e0 + n, None, None]
        if fmt == "fp8_block":
            q, s = _quantize(w.view(n * rows, cols), 128)
            codes.append(q.view(torch.uint8).view(n, rows, cols))
            scales.append(s.view(n, rows // 128, cols // 128))
            continue
        b = w.view(n, rows, cols // (16 if fmt == "nvfp4" else 32), -1)
        amax = b.abs().amax(-1, keepdim=True)
        if fmt == "nvfp4":
            s2 = w.abs().amax((1, 2)) / 2688.0
            sc = (amax / (6.0 * s2[:, None, None, None])).clamp(max=448.0).to(torch.float8_e4m3fn)
            y = b / (sc.float() * s2[:, None, None, None]).clamp(min=1e-30)
            s2s.append(s2)
            scales.append(sc.view(torch.uint8)[..., 0])
        else:
            ex = torch.ceil(torch.log2(amax / (448.0 if fmt == "mxfp8" else 6.0))).clamp(-127, 127)
            y = b / torch.exp2(ex)
            scales.append((ex[..., 0] + 127).to(torch.uint8))
        if fmt == "mxfp8":
            codes.append(y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(n, rows, cols))
        else:
            nib = (torch.bucketize(y.abs(), edges, out_int32=True) + 8 * (y < 0)).to(torch.uint8).view(n, rows, cols // 2, 2)
            codes.append(nib[..., 0] | (nib[..., 1] << 4))
    return torch.cat(codes), torch.cat(scales), (torch.cat(s2s) if s2s else None)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case, status=torch.zeros(1, dtype=torch.int32, device=DEV))
    if case["op"] == "quantize":
        rows, cols, brows = case["rows"], case["cols"], case["brows"]
        s["x"] = _tokens(rows, cols, g) if brows == 1 else (
            torch.randn((rows, cols), generator=g, device=DEV) * 0.02).to(torch.bfloat16)
        s["codes"] = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((-(-rows // brows), -(-cols // 128)), dtype=torch.float32, device=DEV)
    elif case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        a, s["a_scales"] = _quantize(_tokens(m, k, g), 1)
        b, s["b_scales"] = _quantize(torch.randn((n, k), generator=g, device=DEV) * 0.02, 128)
        s["a"], s["b"] = a.view(torch.uint8), b.view(torch.uint8)
        s["c"] = torch.empty((m, n), dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device=DEV)
    else:
        t, e, h, i = case["tokens"], case["experts"], case["hidden"], case["inter"]
        std = torch.exp(torch.empty(e, device=DEV).uniform_(math.log(0.005), math.log(0.05), generator=g))
        s["gate_up"] = _experts(e, 2 * i, h, case["fmt"], std, g)
        s["down"] = _experts(e, h, i, case["fmt"], std, g)
        s["x"] = _tokens(t, h, g)
        top = torch.randn((t, e), generator=g, device=DEV).topk(case["topk"], 1)
        s["ids"] = top.indices.to(torch.int32).contiguous()
        s["weights"] = torch.softmax(top.values, 1).contiguous()
        if case["padded"]:   # rows of the batch that hold no token
            s["ids"][-case["padded"]:] = -1
        s["y"] = torch.empty((t, h), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------- plain forms --
def _decode(codes, scales, s2, fmt):
    """fp32 values of stacked weights (one leading index) from codes and scales."""
    if fmt == "fp8_block":
        return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, 1).repeat_interleave(128, 2)
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
        v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    n, rows, cols = v.shape
    if fmt == "nvfp4":
        d = scales.view(torch.float8_e4m3fn).float() * s2[:, None, None]
    else:
        d = torch.where(scales > 0, (scales.int() << 23).view(torch.float32), 2.0 ** -127)
    return (v.view(n, rows, d.shape[2], -1) * d[..., None]).view(n, rows, cols)


def _pick(stack, at):
    return tuple(None if v is None else v[at] for v in stack)


def _plain_moe(s):
    t, k, h = s["tokens"], s["topk"], s["hidden"]
    ids = s["ids"].view(-1)
    at = ids.clamp(min=0).long()
    x = s["x"].float().repeat_interleave(k, 0)
    gu = torch.matmul(_decode(*_pick(s["gate_up"], at), s["fmt"]), x[:, :, None])[:, :, 0]
    g, u = gu.chunk(2, 1)
    z = torch.matmul(_decode(*_pick(s["down"], at), s["fmt"]), (g * torch.sigmoid(g) * u)[:, :, None])[:, :, 0]
    z = torch.where(ids[:, None] >= 0, z * s["weights"].view(-1, 1), 0.0)
    return z.view(t, k, h).sum(1).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        from mxfp_block_scaled_b200 import mxq
        if s["op"] == "quantize":
            mxq.mxq_quantize_fp8(s["x"], s["rows"], s["cols"], s["brows"], 128, s["codes"], s["scales"], s["status"])
            return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
        if s["op"] == "gemm":
            mxq.mxq_gemm_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"], s["m"], s["n"], s["k"], s["out"], s["c"],
                             s["status"])
            return {"c": s["c"]}
        if "workspace" not in s:   # kept by the caller from call to call
            s["workspace"] = mxq.moe_workspace(s["tokens"], s["topk"], s["hidden"], s["inter"], s["x"].device)
        mxq.mxq_moe_forward(s["x"], s["tokens"], s["hidden"], s["ids"], s["weights"], s["topk"], s["fmt"], s["experts"],
                            s["inter"], *s["gate_up"], *s["down"], s["y"], s["status"], s["workspace"])
        return {"y": s["y"]}
    if s["op"] == "quantize":
        codes, scales = _quantize(s["x"], s["brows"])
        return {"codes": codes, "scales": scales}
    if s["op"] == "gemm":
        a = s["a"].view(torch.float8_e4m3fn).float() * _spread(s["a_scales"], 1, s["m"], s["k"])
        b = s["b"].view(torch.float8_e4m3fn).float() * _spread(s["b_scales"], 128, s["n"], s["k"])
        return {"c": torch.matmul(a, b.t()).to(s["c"].dtype)}
    return {"y": _plain_moe(s)}


# -------------------------------------------------------------- definition --
def _e4m3_values():
    """The value of each E4M3 byte, from its fields."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(math.nan if c & 127 == 127 else -x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _values64(stack, e, fmt, e4m3):
    """One expert's weights in binary64."""
    codes, scales, s2 = stack
    if fmt in ("nvfp4", "mxfp4"):
        grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
        n = torch.stack((codes[e] % 16, codes[e].div(16, rounding_mode="floor")), -1).reshape(codes.shape[1], -1).long()
        v = grid[n % 8] * (1 - 2 * (n // 8)).double()
    else:
        v = e4m3[codes[e].long()]
    if fmt == "fp8_block":
        r, c = (torch.arange(x, device=DEV) // 128 for x in v.shape)
        return v * scales[e].double()[r[:, None], c[None, :]]
    if fmt == "nvfp4":
        d = e4m3[scales[e].long()] * s2[e].double()
    else:
        d = torch.ldexp(torch.ones_like(scales[e], dtype=torch.float64), scales[e].long() - 127)
    return v * d[:, torch.arange(v.shape[1], device=DEV) // (v.shape[1] // d.shape[1])]


def exact(case, seed):
    s = prepare(case, seed)
    e4m3 = _e4m3_values()
    if case["op"] == "quantize":
        x, br = s["x"].double(), case["brows"]
        rows, cols = x.shape
        scale = torch.zeros((-(-rows // br), -(-cols // 128)), dtype=torch.float64, device=DEV)
        for b in range(scale.shape[1]):
            a = x[:, 128 * b:128 * b + 128].abs().amax(1)
            idx = torch.arange(rows, device=DEV) // br
            scale[:, b] = torch.zeros(scale.shape[0], dtype=torch.float64, device=DEV).scatter_reduce(0, idx, a, "amax") / 448.0
        return {"codes": None, "scales": scale}   # codes are whole choices: a value next to a border may go either way
    if case["op"] == "gemm":
        c = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device=DEV)
        row = torch.arange(case["n"], device=DEV) // 128
        for kb in range(s["a_scales"].shape[1]):
            cut = slice(128 * kb, 128 * kb + 128)
            a = e4m3[s["a"][:, cut].long()] * s["a_scales"][:, kb, None].double()
            b = e4m3[s["b"][:, cut].long()] * s["b_scales"][row, kb, None].double()
            c.addmm_(a, b.t())
        return {"c": c}
    y = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device=DEV)
    for e in sorted(set(s["ids"].view(-1).tolist()) - {-1}):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        g, u = (s["x"][t].double() @ _values64(s["gate_up"], e, case["fmt"], e4m3).t()).chunk(2, 1)
        z = (g / (1.0 + torch.exp(-g)) * u) @ _values64(s["down"], e, case["fmt"], e4m3).t()
        y.index_add_(0, t, z * s["weights"][t, j, None].double())
    return {"y": y}


# -------------------------------------------------------------------- work --
def work(case):
    if case["op"] == "quantize":
        n, nb = case["rows"] * case["cols"], -(-case["rows"] // case["brows"]) * -(-case["cols"] // 128)
        return {"bytes": 3 * n + 4 * nb, "flops": 2 * n}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // 128)
        return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // 128)) + m * n * (4 if case["out"] == "f32" else 2),
                "flops": 2 * m * n * k}
    t = case["tokens"] - case["padded"]
    e, h, i = case["experts"], case["hidden"], case["inter"]
    distinct = e * (1.0 - (1.0 - case["topk"] / e) ** t)   # experts that at least one of the tokens chose, on average
    per = {"nvfp4": 0.5 + 1 / 16, "mxfp4": 0.5 + 1 / 32, "mxfp8": 1 + 1 / 32, "fp8_block": 1 + 4 / 16384}[case["fmt"]]
    return {"bytes": distinct * 3 * i * h * per + case["tokens"] * (4 * h + 8 * case["topk"]),
            "flops": 6 * t * case["topk"] * i * h}

"""Attention over the quantized cache where its numbers reach far: scores whose neighbours in
fp32 lie 16 apart, weights far below the largest.

Bounds as in test_gpu_cache_attention.py, without its allowance for what lies far below the
largest term.  In its place, of weights: they are rounded to f16, whose step below its normal
numbers is 2^-24, and the largest one of a row stands at 2^7 or above, so each is off by 2^-32
of the largest at most."""
import math

import numpy as np
import pytest
import torch

import cache_ref as ref
from mxfp_block_scaled_b200 import mxq
from test_gpu_cache import dev32, gen
from test_gpu_cache_attention import filled

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950408889634


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def one_sequence(fmt, n, dim, tokens=64, heads=1):
    """A cache whose one sequence holds n tokens, its pages in order, codes 0."""
    pages = -(-n // tokens)
    s2 = (torch.ones(heads, device="cuda"),) * 2 if fmt == "nvfp4" else (None, None)
    cache = mxq.Cache.empty(pages, heads, tokens, dim, fmt, *s2)
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(127 if fmt == "mxfp8" else 0x38)        # 1
    return cache, dev32([n]), torch.arange(pages, dtype=torch.int32, device="cuda")[None]


def rows_of(t, n):
    """The n tokens of a cache tensor [pages, 1, tokens, width] in order, a view."""
    return t.view(-1, t.shape[-1])[:n]


def attend(cache, q, ln, table, scale):
    new = q.shape[0]
    r = mxq.cache_attention(cache, q, dev32([0, new]), ln, table, new, scale=scale)
    assert r["status"].item() == 0
    return r


def check(r, cache, q, ln, table, scale, more=0.0):
    """Every output and lse; `more`: a further allowance of outputs."""
    cu = [0, q.shape[0]]
    o, lse, weight, spread = ref.attention(cache, q, cu, ln.tolist(), table, scale)
    eps = 2 * (cache.head_dim + 8) * 2.0 ** -23 * spread
    largest = largest_weight(cache, q, ln, table, scale, lse)
    size = ref.sequence_values(cache, 0, ln, table)[1].abs().amax(0)        # [1, dim], of a column
    bound = 1.01 * (o.abs() * 2.0 ** -8 + weight * (2.0 ** -11 + eps[..., None] + 2.0 ** -18) * (1 + 2.0 ** -8)) \
        + int(ln[0]) * 2.0 ** -32 * largest[..., None] * size + more + 1e-30
    worst = ((r["o"].double() - o).abs() / bound).max().item()
    assert worst <= 1, worst
    off = ((r["lse"].double() - lse).abs() / (eps + 2.0 ** -18 + lse.abs() * 2.0 ** -22)).max().item()
    assert off <= 1, off


def largest_weight(cache, q, ln, table, scale, lse):
    """The largest softmax weight of each row, [T, heads]."""
    k = ref.sequence_values(cache, 0, ln, table)[0][:, 0]
    new = q.shape[0]
    s = scale * torch.einsum("ihd,jd->ihj", q.double(), k)
    pos = int(ln[0]) - new + torch.arange(new, device=q.device)
    s.masked_fill_((torch.arange(k.shape[0], device=q.device)[None] > pos[:, None])[:, None], -math.inf)
    return torch.exp(s.amax(-1) - lse)


def scale_with(bits):
    """An fp32 scale whose fp32 product with log2(e) has these last bits of 2^27."""
    want = np.float32(2.0 ** 27 * (1 + bits * 2.0 ** -23))
    at = np.float32(float(want) / LOG2E)
    for _ in range(8):
        at = np.nextafter(at, np.float32(0))
    for _ in range(16):
        if np.float32(at * np.float32(LOG2E)) == want:
            return float(at)
        at = np.nextafter(at, np.float32(np.inf))
    return None


@pytest.mark.parametrize("new", [1, 80])
@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_scores_whose_neighbours_lie_sixteen_apart(fmt, new):
    """Scores 2^27 (1 + n 2^-23), in powers of two: the next larger one after the largest so
    far is 2^16 times the weight, whatever the last bit of either.  Outputs lie between the
    values and go with the largest."""
    n, dim = 4096, 64
    cache, ln, table = one_sequence(fmt, n, dim)
    k, v = rows_of(cache.k_codes, n), rows_of(cache.v_codes, n)
    later = torch.arange(n, device="cuda") // 128 % 2 == 1        # (whoever has 256 neighbours sees both)
    if fmt == "mxfp8":                          # k = (1, 0 or 2^-6 in dimension 32), v = 1 or 2
        k[:, 0] = 0x38
        k[:, 32] = torch.where(later, 0x08, 0).to(torch.uint8)
        v[:] = torch.where(later, 0x40, 0x38).to(torch.uint8)[:, None]
    else:                                       # the same, the second block's scale 2^-6
        k[:, 0] = 0x02
        k[:, 16] = torch.where(later, 0x02, 0).to(torch.uint8)
        rows_of(cache.k_scales, n)[:, 2] = 0x08
        v[:] = torch.where(later, 0x44, 0x22).to(torch.uint8)[:, None]
    q = torch.zeros((new, 2, dim), dtype=torch.bfloat16, device="cuda")
    q[..., 0], q[..., 32] = 1.0, 2.0 ** -17     # 2^-23 of the first product
    found = 0
    for bits in range(1, 24):
        scale = scale_with(bits)
        if scale is None:
            continue
        found += 1
        r = attend(cache, q, ln, table, scale)
        # (one key with a score between may be what the sum's last bit makes of it)
        assert torch.isfinite(r["o"].float()).all() and torch.isfinite(r["lse"]).all(), bits
        assert (r["o"].float() >= 1).all() and (r["o"].float() <= 2).all(), bits
    assert found >= 4


@pytest.mark.parametrize("new", [1, 5, 80])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_scores_of_any_size(fmt, dim, new):
    """Scores up to 2^60 that are no round numbers: a product rounded in one place and not in
    another would leave weights without bound.  Outputs lie between the values."""
    cache, ln, table = filled(fmt, [3000], 1, 32, dim, 17, spread=0)
    q = torch.randn((new, 4, dim), generator=gen(5), device="cuda").bfloat16()
    v = ref.sequence_values(cache, 0, ln, table)[1].abs().amax()
    for power in (20, 24, 25, 26, 27, 28, 29, 30, 33, 40, 57):
        for scale in (1.37 * 2.0 ** power, -1.61 * 2.0 ** power):
            r = attend(cache, q, ln, table, scale)
            assert torch.isfinite(r["lse"]).all() and (r["o"].double().abs() <= v * (1 + 2.0 ** -8)).all(), scale


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("every", [1 << 30, 32])
@pytest.mark.parametrize("below", [16.3, 22.7, 24.6, 26.2])
@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_weights_far_below_the_largest(fmt, below, every, new):
    """A first token that takes the weight (or one in 32 tokens) and has no value, and many whose
    weights are 2^-below of its: the output is theirs."""
    n, dim = 1 << 18, 64
    cache, ln, table = one_sequence(fmt, n, dim)
    k, v = rows_of(cache.k_codes, n), rows_of(cache.v_codes, n)
    sink = torch.arange(n, device="cuda") % every == 0
    one = 0x38 if fmt == "mxfp8" else 0x02
    k[:, 0] = torch.where(sink, one, 0).to(torch.uint8)
    codes = torch.tensor([0x38, 0x3C, 0x40, 0x30] if fmt == "mxfp8" else [0x22, 0x33, 0x44, 0x21], device="cuda", dtype=torch.uint8)
    v[:] = codes[torch.randint(0, 4, v.shape, generator=gen(1), device="cuda")]
    v[sink] = 0
    q = torch.zeros((new, 1, dim), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = below / LOG2E
    check(attend(cache, q, ln, table, scale), cache, q, ln, table, scale)

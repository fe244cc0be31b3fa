"""Attention over sequences of millions of tokens, whose pages repeat (a page that sequences or
places share is for reading), against binary64 over the distinct tokens and how often each is
seen: sums over all of a tile's keys by one CTA.

Bounds as in test_gpu_attention_numerics.py, and 2^-12 for sums of products that are cut to fp32
in pieces of 2^15 keys: a cut each 16 keys, of at most 2^-23 of the sum so far, which grows
evenly, so half of 2^11 2^-23."""
import math

import pytest
import torch

import cache_ref as ref
from mxfp_block_scaled_b200 import mxq
from test_gpu_cache import dev32, gen

pytestmark = pytest.mark.gpu
PAGES, TOKENS = 64, 256         # distinct


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def repeating(fmt, dim):
    s2 = (torch.ones(1, device="cuda"),) * 2 if fmt == "nvfp4" else (None, None)
    cache = mxq.Cache.empty(PAGES, 1, TOKENS, dim, fmt, *s2)
    rand = lambda lo, hi, t, s: torch.randint(lo, hi, t.shape, device="cuda", generator=gen(s))  # noqa: E731
    if fmt == "mxfp8":          # values from 0.5 to 1.9, keys from 0 to 0.5
        cache.v_codes.copy_(rand(0x30, 0x40, cache.v_codes, 1))
        cache.k_codes.copy_(rand(0, 0x30, cache.k_codes, 2))
    else:
        cache.v_codes.copy_(rand(1, 8, cache.v_codes, 1) + 16 * rand(1, 8, cache.v_codes, 2))
        cache.k_codes.copy_(rand(1, 8, cache.k_codes, 3) + 16 * rand(1, 8, cache.k_codes, 4))
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(127 if fmt == "mxfp8" else 0x38)
    return cache


def check_row(o, lse, q, cache, pos, scale):
    """Of one row: q [heads, dim], which sees the positions up to pos."""
    n = PAGES * TOKENS
    s2 = None if cache.k_s2 is None else torch.ones(n, device="cuda")
    k, v = (ref.values(c.view(n, -1), s.view(n, -1), cache.fmt, s2)
            for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)))
    seen = (pos + 1) // n + (torch.arange(n, device="cuda") < (pos + 1) % n).double()
    s = scale * q.double() @ k.t()
    want_lse = torch.logsumexp(s + seen.log(), -1)
    p = seen * torch.exp(s - want_lse[:, None])
    want = p @ v
    eps = 2 * (cache.head_dim + 8) * 2.0 ** -23 * scale * (q.double().abs() @ k.abs().t()).amax(-1)
    largest = torch.exp(s - want_lse[:, None]).amax(-1)
    bound = 1.01 * (want * 2.0 ** -8 + want * (2.0 ** -11 + 2.0 ** -12 + eps[:, None] + 2.0 ** -18) * (1 + 2.0 ** -8)) \
        + (pos + 1) * 2.0 ** -32 * largest[:, None] * v.max()
    worst = ((o.double() - want).abs() / bound).max().item()
    assert worst <= 1, worst
    assert ((lse.double() - want_lse).abs() <= eps + 2.0 ** -16 + want_lse.abs() * 2.0 ** -22).all()
    # the mean of the errors is no bias: rows and columns many times over
    assert abs(((o.double() - want) / want).mean().item()) < 2.0 ** -11


@pytest.mark.parametrize("fmt,dim", [("mxfp8", 64), ("nvfp4", 64), ("mxfp8", 128), ("nvfp4", 256)])
def test_a_chunk_over_millions_of_tokens(fmt, dim):
    """160 tiles of 256 rows (320 of 128) over 4 194 304 tokens: a CTA has whole tiles."""
    n, new, group, scale = 1 << 22, 160, 256, 0.05
    cache = repeating(fmt, dim)
    table = (torch.arange(n // TOKENS, device="cuda") % PAGES).int()[None]
    q = torch.randn((new, group, dim), device="cuda", generator=gen(9)).bfloat16()
    r = mxq.cache_attention(cache, q, dev32([0, new]), dev32([n]), table, new, scale=scale)
    assert r["status"].item() == 0
    for row in (0, 1, 77, 159):
        check_row(r["o"][row], r["lse"][row], q[row], cache, n - new + row, scale)


@pytest.mark.parametrize("fmt,dim,group,seqs", [("mxfp8", 64, 8, 800), ("nvfp4", 128, 16, 600), ("mxfp8", 256, 4, 300)])
def test_decoding_over_millions_of_tokens(fmt, dim, group, seqs):
    """More sequences of 2 097 152 tokens than CTAs, on the same pages."""
    n, scale = 1 << 21, 0.05
    cache = repeating(fmt, dim)
    table = (torch.arange(n // TOKENS, device="cuda") % PAGES).int()[None].expand(seqs, -1).contiguous()
    lens = [n - 1000 * b for b in range(seqs)]
    q = torch.randn((seqs, group, dim), device="cuda", generator=gen(9)).bfloat16()
    r = mxq.cache_attention(cache, q, dev32(range(seqs + 1)), dev32(lens), table, 1, scale=scale)
    assert r["status"].item() == 0
    for row in (0, 1, 100, seqs // 2, seqs - 1):
        check_row(r["o"][row], r["lse"][row], q[row], cache, lens[row] - 1, scale)

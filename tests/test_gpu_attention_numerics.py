"""Attention over the quantized cache where its numbers reach far: scores whose neighbours in
fp32 lie 16 apart."""
import numpy as np
import pytest
import torch

from mxfp_block_scaled_b200 import mxq
from test_gpu_cache import dev32, gen

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

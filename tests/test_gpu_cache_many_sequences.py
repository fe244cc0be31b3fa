"""Calls on a cache with as many sequences as they take: more than a CTA has threads."""
import pytest
import torch

from mxfp_block_scaled_b200 import mxq
from test_gpu_cache import dev32, gen, make_cache
from test_gpu_cache_attention import check, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def sums(v):
    out = [0]
    for n in v:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("seqs,most_new,longest,heads,group,dim", [
    (129, 1, 400, 2, 4, 128), (513, 3, 60, 1, 2, 64), (1000, 1, 40, 4, 8, 64), (4096, 1, 50, 1, 1, 128), (4095, 2, 20, 2, 9, 256),
    (600, 70, 200, 1, 1, 64), (300, 90, 300, 2, 2, 128), (4096, 80, 90, 1, 1, 64)])
def test_attention(seqs, most_new, longest, heads, group, dim, fmt):
    """Some of no token, some of no new one; chosen ones against binary64, all against calls of a part."""
    r = torch.Generator().manual_seed(seqs)
    lens = torch.randint(0, longest + 1, (seqs,), generator=r)
    news = torch.minimum(torch.randint(0, most_new + 1, (seqs,), generator=r), lens)
    news[-1] = lens[-1] = most_new
    lens, news = lens.tolist(), news.tolist()
    cache, ln, table = filled(fmt, lens, heads, 16, dim, seqs)
    cu = sums(news)
    q = torch.randn((cu[-1] + 2, heads * group, dim), generator=gen(2), device="cuda").bfloat16()
    got = mxq.cache_attention(cache, q, dev32(cu), ln, table, most_new)
    assert got["status"].item() == 0 and (got["o"][cu[-1]:] == 0).all()
    assert torch.equal(got["o"], mxq.cache_attention(cache, q, dev32(cu), ln, table, most_new)["o"])
    for b in [0, 1, 127, 128, seqs // 2, seqs - 2, seqs - 1]:
        rows = slice(cu[b], cu[b + 1])
        if news[b]:
            check({"o": got["o"][rows], "lse": got["lse"][rows]}, cache, q[rows], dev32([0, news[b]]), ln[b:b + 1], table[b:b + 1], dim ** -0.5)
    # parts of 100 sequences: other divisions of the work, the same within two roundings
    for b in range(0, seqs, 100):
        e = min(b + 100, seqs)
        if cu[e] > cu[b]:
            part = mxq.cache_attention(cache, q[cu[b]:cu[e]], dev32([x - cu[b] for x in cu[b:e + 1]]), ln[b:e], table[b:e].contiguous(), most_new)
            x, y = got["o"][cu[b]:cu[e]].float(), part["o"].float()
            limit = 2.0 ** -7 * torch.maximum(x.abs(), y.abs()) + 2.0 ** -5     # (2^-11 of sums of |v| below 16, twice, and the rounding)
            assert ((x - y).abs() <= limit).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("seqs", [33, 1000, 1025, 4096])
def test_write_and_read(seqs, fmt):
    r = torch.Generator().manual_seed(seqs)
    lens = torch.randint(0, 40, (seqs,), generator=r)
    news = torch.minimum(torch.randint(0, 6, (seqs,), generator=r), lens)
    cu = sums(news.tolist())
    pages = sum(-(-n // 16) for n in lens.tolist())
    cache, order, at = make_cache(fmt, pages, 1, 16, 64), torch.randperm(pages, generator=r), 0
    table = torch.full((seqs, 3), -1, dtype=torch.int32)
    for b, n in enumerate(lens.tolist()):
        need = -(-n // 16)
        table[b, :need] = order[at:at + need]
        at += need
    table, ln, T = table.cuda(), dev32(lens.tolist()), cu[-1] + 3
    k, v = (torch.randn((T, 1, 64), generator=gen(i), device="cuda").bfloat16() for i in range(2))
    assert mxq.cache_write(cache, k, v, dev32(cu), ln, table).item() == 0
    whole = mxq.cache_read(cache, dev32(cu), ln, table, T)
    assert whole["status"].item() == 0 and (whole["k"][cu[-1]:] == 0).all()
    for b in range(0, seqs, 31):        # a few sequences alone, into a cache of their own
        e = min(b + 31, seqs)
        if cu[e] == cu[b]:
            continue
        one, rows = make_cache(fmt, pages, 1, 16, 64), slice(cu[b], cu[e])
        part = dev32([x - cu[b] for x in cu[b:e + 1]]), ln[b:e], table[b:e].contiguous()
        assert mxq.cache_write(one, k[rows], v[rows], *part).item() == 0
        back = mxq.cache_read(one, *part, cu[e] - cu[b])
        assert torch.equal(back["k"], whole["k"][rows]) and torch.equal(back["v"], whole["v"][rows])


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("heads,group,dim,news,lens", [
    (1024, 1, 64, [3, 1], [50, 20]), (1000, 2, 256, [1, 1], [40, 17]), (257, 3, 128, [2, 70], [90, 200]), (1, 256, 128, [1, 3], [500, 70]),
    (3, 256, 64, [1], [2000])])
def test_as_many_heads_as_there_may_be(heads, group, dim, news, lens, fmt):
    cache, ln, table = filled(fmt, lens, heads, 16, dim, heads)
    cu = dev32(sums(news))
    back = mxq.cache_read(cache, cu, ln, table, sum(news))
    q = torch.randn((sum(news), heads * group, dim), generator=gen(2), device="cuda").bfloat16()
    r = mxq.cache_attention(cache, q, cu, ln, table, max(news))
    assert back["status"].item() == 0 and r["status"].item() == 0
    check(r, cache, q, cu, ln, table, dim ** -0.5)
    # the last tokens written again from what was read: the values of their codes once more
    again, _, _ = filled(fmt, lens, heads, 16, dim, heads)
    mxq.cache_write(again, back["k"], back["v"], cu, ln, table)
    if fmt == "mxfp8":
        assert torch.equal(mxq.cache_read(again, cu, ln, table, sum(news))["v"], back["v"])

"""Attention over the quantized cache at the lengths that it is used at: chunks of prompts in
which a CTA goes through tens of steps and several tiles (its rings of buffers many times over),
of two groups of rows and of one, on pages of every size; decoding whose work is divided with many
turns of a warp; both in one batch.  Against binary64, bounds as in test_gpu_cache_attention.py."""
import pytest
import torch

from mxfp_block_scaled_b200 import mxq
from test_gpu_cache import dev32, gen
from test_gpu_cache_attention import check, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def rising(q, news):
    """Queries that grow along each sequence's rows, so that maxima lie anywhere."""
    at = torch.cat([torch.linspace(0.2, 3.0, max(n, 1))[:n] for n in news]).to(q.device)
    return (q.float() * at[:, None, None]).bfloat16()


def run(fmt, news, lens, heads, group, tokens, dim, most=None):
    cache, ln, table = filled(fmt, lens, heads, tokens, dim, sum(lens))
    cu = dev32([sum(news[:i]) for i in range(len(news) + 1)])
    q = rising(torch.randn((sum(news), heads * group, dim), generator=gen(7), device="cuda"), news)
    r = mxq.cache_attention(cache, q, cu, ln, table, most or max(news))
    assert r["status"].item() == 0
    again = mxq.cache_attention(cache, q, cu, ln, table, most or max(news))
    assert torch.equal(r["o"], again["o"]) and torch.equal(r["lse"], again["lse"])
    # a sequence at a time (the reference's matrices are large)
    for b, (n, length) in enumerate(zip(news, lens)):
        rows = slice(sum(news[:b]), sum(news[:b]) + n)
        if n:
            part = {"o": r["o"][rows], "lse": r["lse"][rows]}
            check(part, cache, q[rows], dev32([0, n]), ln[b:b + 1], table[b:b + 1], dim ** -0.5)


CHUNKS = [
    # new, in all, kv heads, query heads to one, page, dim.  Steps of a CTA (of 64 keys): 40 to 90
    ([600, 130, 40, 65, 900], [4000, 2500, 5000, 70, 3000], 8, 4, 64, 128),
    ([300, 1, 17, 260], [9000, 3000, 700, 2000], 8, 8, 16, 64),
    ([500], [6000], 8, 8, 32, 256),
    ([70, 70, 70, 70, 70, 70, 70, 70], [3000, 200, 2500, 64, 128, 70, 4000, 1000], 16, 2, 128, 128),      # one group: 140 rows, 2
    ([100] * 12, [7000 - 500 * i for i in range(12)], 8, 1, 256, 128),                                    # one group alone
    ([2048], [2048], 8, 4, 64, 64),                                                                       # a prompt from its beginning
    ([130, 64, 3, 900], [8000, 9000, 100, 900], 4, 3, 16, 256)]


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("news,lens,heads,group,tokens,dim", CHUNKS)
def test_chunks_of_many_steps(fmt, news, lens, heads, group, tokens, dim):
    run(fmt, news, lens, heads, group, tokens, dim)


DECODING = [
    # turns of a warp: 10 to 40; tiles of 8 and of 16 rows, one and several a sequence
    ([1] * 16, [20000 - 1111 * i for i in range(16)], 8, 4, 64, 128), ([1] * 24, [9000 + 100 * i for i in range(24)], 4, 8, 16, 64),
    ([2] * 8, [20000 - 999 * i for i in range(8)], 4, 8, 32, 256), ([4, 1, 0, 3] * 6, [9000, 16000, 5, 30000] * 6, 2, 8, 128, 128),
    ([1] * 40, [4096] * 40, 8, 1, 256, 256)]


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("news,lens,heads,group,tokens,dim", DECODING)
def test_decoding_of_many_turns(fmt, news, lens, heads, group, tokens, dim):
    run(fmt, news, lens, heads, group, tokens, dim)


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("dim,group", [(128, 8), (64, 3), (256, 4)])
def test_a_chunk_beside_decoding(fmt, dim, group):
    """A batch as a server has it: one sequence with a chunk of its prompt, the others with a token,
    some with guessed ones."""
    news = [1, 1, 5, 700, 1, 0, 1, 3] + [1] * 20
    lens = [3000, 1, 900, 2500, 17, 40, 8000, 64] + [1000 + 77 * i for i in range(20)]
    run(fmt, news, lens, 4, group, 64, dim)

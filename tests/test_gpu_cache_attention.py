"""Attention over the quantized cache on the GPU against binary64 over the same codes.

Bound of an output element, relative to sum_j p_j |v_j|: weights are rounded to 11 bits
(2^-11) against a sum of unrounded ones; a score is off by the fp32 sum of dim products,
cut rather than rounded ((dim + 8) 2^-23 of scale sum |q k|), once in a weight and once in
the sum; exponentials and the running rescaling add 2^-18; MXFP8 codes far below a
neighbour's and weights below f16's normal numbers add keys 2^-25 of the largest term.  The
result is then rounded to bf16 (2^-8)."""
import math
import threading

import pytest
import torch

import cache_ref as ref
from mxfp_block_scaled_b200 import layers, mxq
from test_gpu_cache import batch, dev32, gen, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def filled(fmt, lens, heads, tokens, dim, seed, spread=2, pages=None):
    """A cache with every sequence's tokens in it, NaN patterns elsewhere, and its table."""
    pages = pages or sum(-(-n // tokens) for n in lens) + 1
    cache = make_cache(fmt, pages, heads, tokens, dim, seed, fill=0x7F if fmt == "mxfp8" else 0xFF)
    if fmt == "nvfp4":
        cache.k_s2.fill_(1 / 256), cache.v_s2.copy_(torch.linspace(0.002, 0.01, heads, device="cuda"))
        cache.k_scales.fill_(0x7F), cache.v_scales.fill_(0xFF)
    else:
        cache.k_scales.fill_(0xFF), cache.v_scales.fill_(0xFE)
    cu, ln, table = batch(lens, lens, tokens, pages, seed)
    k, v = (torch.randn((sum(lens), heads, dim), generator=gen(seed + i), device="cuda") for i in range(2))
    v *= torch.exp2(torch.randint(-spread, spread + 1, (sum(lens), heads, 1), generator=gen(seed + 2), device="cuda").float())
    mxq.cache_write(cache, k.bfloat16(), v.bfloat16(), cu, ln, table)
    return cache, ln, table


def check(got, cache, q, cu, ln, table, scale, rows=None):
    o, lse, weight, spread = ref.attention(cache, q, cu.tolist(), ln.tolist(), table, scale)
    keys = max(ln.tolist() + [1])
    eps = 2 * (cache.head_dim + 8) * 2.0 ** -23 * spread
    term = weight.amax((1, 2), keepdim=True)
    bound = 1.01 * (o.abs() * 2.0 ** -8 + weight * (2.0 ** -11 + eps[..., None] + 2.0 ** -18) * (1 + 2.0 ** -8)) \
        + term * keys * 2.0 ** -25 + 1e-30
    rows = slice(None) if rows is None else rows
    worst = ((got["o"].double() - o).abs() / bound)[rows].max().item()
    assert worst <= 1, worst
    seen = lse > -math.inf
    assert torch.equal(got["lse"][rows] == -math.inf, ~seen[rows])
    tol = eps + 2.0 ** -18 + lse.abs() * 2.0 ** -22
    off = torch.where(seen, (got["lse"].double() - lse).abs() / tol, 0.0)[rows].max().item()
    assert off <= 1, off


SHAPES = [
    # new, in all, kv heads, query heads to one, page, dim
    ([1], [1], 1, 1, 16, 64), ([1], [5000], 2, 8, 64, 128), ([1, 1, 1], [70, 1, 513], 2, 4, 16, 256), ([1] * 40, list(range(1, 2400, 60)), 1, 5, 32, 128),
    ([4, 3, 0, 1], [100, 3, 50, 2000], 2, 8, 32, 128), ([6], [900], 3, 7, 128, 64), ([64, 1], [64, 1], 1, 1, 16, 64),
    ([65], [65], 2, 1, 16, 128), ([100, 17, 1, 5], [300, 17, 1025, 700], 2, 8, 64, 128), ([333], [1000], 1, 3, 256, 256),
    ([40, 200], [41, 999], 2, 13, 16, 64), ([600], [600], 1, 16, 128, 128), ([1], [40001], 1, 2, 256, 64), ([2, 130], [9000, 300], 1, 256, 64, 64)]


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("news,lens,heads,group,tokens,dim", SHAPES)
def test_against_binary64(fmt, news, lens, heads, group, tokens, dim):
    cache, ln, table = filled(fmt, lens, heads, tokens, dim, sum(lens))
    T = sum(news) + 3
    cu = dev32([1] + [1 + sum(news[:i + 1]) for i in range(len(news))])
    wide = torch.randn((T, heads * group + 2, dim), generator=gen(T), device="cuda").bfloat16()
    q = wide[:, 1:-1]           # strided
    r = mxq.cache_attention(cache, q, cu, ln, table, max(news))
    check(r, cache, q, cu, ln, table, dim ** -0.5)
    assert r["status"].item() == 0 and (r["o"][0] == 0).all() and (r["o"][-2:] == 0).all() and (r["lse"][-2:] == 0).all()
    again = mxq.cache_attention(cache, q, cu, ln, table, max(news))
    assert torch.equal(r["o"], again["o"]) and torch.equal(r["lse"], again["lse"])
    # a looser bound on the rows may take another way through, not to other values
    check(mxq.cache_attention(cache, q, cu, ln, table, 100000), cache, q, cu, ln, table, dim ** -0.5)


@pytest.mark.parametrize("fmt,dim", [("mxfp8", 128), ("nvfp4", 64)])
@pytest.mark.parametrize("new,group", [(3, 4), (90, 2)])
def test_rows_without_a_key(fmt, dim, new, group):
    """A sequence of fewer tokens than rows, one of none, beside an ordinary one."""
    lens = [2, 0, 77]
    cache, ln, table = filled(fmt, lens, 2, 16, dim, 5)
    cu = dev32([0, new, 2 * new, 3 * new])
    q = torch.randn((3 * new, 2 * group, dim), generator=gen(1), device="cuda").bfloat16()
    r = mxq.cache_attention(cache, q, cu, ln, table, new)
    check(r, cache, q, cu, ln, table, dim ** -0.5)
    assert (r["o"][:new - 2] == 0).all() and (r["o"][new:2 * new] == 0).all() and r["status"].item() == 0


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0, 1e-30])
@pytest.mark.parametrize("new", [1, 80])
def test_scales(scale, new):
    cache, ln, table = filled("mxfp8", [500], 2, 64, 128, 9)
    q = torch.randn((new, 8, 128), generator=gen(2), device="cuda").bfloat16()
    cu = dev32([0, new])
    check(mxq.cache_attention(cache, q, cu, ln, table, new, scale=scale), cache, q, cu, ln, table, scale)


@pytest.mark.parametrize("new", [1, 80])
@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_queries_and_values_of_very_different_sizes(fmt, new):
    cache, ln, table = filled(fmt, [700], 1, 32, 128, 11, spread=8 if fmt == "mxfp8" else 2)
    q = torch.randn((new, 4, 128), generator=gen(2), device="cuda")
    q *= torch.exp2(torch.tensor([-30.0, -3.0, 0.0, 4.0], device="cuda"))[None, :, None]
    q = q.bfloat16()
    q[0, 2] = 0
    cu = dev32([0, new])
    check(mxq.cache_attention(cache, q, cu, ln, table, new), cache, q, cu, ln, table, 128 ** -0.5)


@pytest.mark.parametrize("new", [1, 5, 80])
@pytest.mark.parametrize("low,high", [(-30, 4), (-90, -60), (30, 60), (60, 90)])
def test_tokens_of_very_different_sizes(new, low, high):
    """MXFP8 scales that lie up to 2^34 apart from one token and block to the next, and far
    from 1; scores of ordinary size, of 2^30 and of 2^60 and more, of both signs."""
    lens, dim = [600], 128
    cache, ln, table = filled("mxfp8", lens, 1, 32, dim, 13)
    g = gen(14)
    k, v = (torch.randn((600, 1, dim // 32, 32), generator=g, device="cuda")
            * torch.exp2(torch.randint(low, high + 1, (600, 1, dim // 32, 1), generator=g, device="cuda").float()) for _ in range(2))
    mxq.cache_write(cache, k.view(600, 1, dim).bfloat16(), v.view(600, 1, dim).bfloat16(), dev32([0, 600]), ln, table)
    q = torch.randn((new, 4, dim), generator=g, device="cuda").bfloat16()
    cu = dev32([0, new])
    for scale in (dim ** -0.5, 2.0 ** -high, 2.0 ** (24 - high), -2.0 ** (24 - high)):
        check(mxq.cache_attention(cache, q, cu, ln, table, new, scale=scale), cache, q, cu, ln, table, scale)


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("new,group", [(1, 4), (3, 8), (150, 2)])
def test_a_nonfinite_query_leaves_the_others(fmt, new, group):
    cache, ln, table = filled(fmt, [900, 400], 1, 16, 128, 3)
    q = torch.randn((2 * new, group, 128), generator=gen(1), device="cuda").bfloat16()
    cu = dev32([0, new, 2 * new])
    want = mxq.cache_attention(cache, q, cu, ln, table, new)
    for bad in (float("nan"), float("inf"), float("-inf")):
        z = q.clone()
        z[new // 2, 1, 77] = bad
        r = mxq.cache_attention(cache, z, cu, ln, table, new)
        keep = torch.ones((2 * new, group), dtype=torch.bool, device="cuda")
        keep[new // 2, 1] = False
        assert torch.equal(r["o"][keep], want["o"][keep]) and torch.equal(r["lse"][keep], want["lse"][keep])
        assert r["status"].item() == 0


@pytest.mark.parametrize("new,group", [(2, 4), (70, 2)])
def test_bad_pages_leave_the_other_sequences(new, group):
    lens = [100, 200, 90, 400]
    cache, ln, table = filled("mxfp8", lens, 2, 16, 128, 3)
    q = torch.randn((4 * new, 2 * group, 128), generator=gen(1), device="cuda").bfloat16()
    cu = dev32([i * new for i in range(5)])
    want = mxq.cache_attention(cache, q, cu, ln, table, new)
    assert want["status"].item() == 0
    for bad in (-1, cache.pages, 1 << 30):
        t = table.clone()
        t[1, 3] = bad
        r = mxq.cache_attention(cache, q, cu, ln, t, new)
        assert r["status"].item() == mxq.DEV_INVALID_PAGE
        keep = torch.cat((torch.arange(new), torch.arange(2 * new, 4 * new))).cuda()
        assert torch.equal(r["o"][keep], want["o"][keep]) and torch.equal(r["lse"][keep], want["lse"][keep])
    # a table that ends before the sequence does
    r = mxq.cache_attention(cache, q[3 * new:], dev32([0, new]), ln[3:], table[3:, :7].contiguous(), new)
    assert r["status"].item() == mxq.DEV_INVALID_PAGE


@pytest.mark.parametrize("new", [1, 90])
def test_a_sequence_longer_than_its_table_is_left_out(new):
    """A length that no table holds costs nothing and leaves the other sequence alone."""
    cache, ln, table = filled("mxfp8", [100, 300], 2, 16, 64, 3)
    q = torch.randn((2 * new, 4, 64), generator=gen(1), device="cuda").bfloat16()
    cu = dev32([0, new, 2 * new])
    for bad in (2 ** 31 - 1, table.shape[1] * 16 + 1):
        r = mxq.cache_attention(cache, q, cu, dev32([bad, 300]), table, new)
        assert r["status"].item() == mxq.DEV_INVALID_PAGE and (r["o"][:new] == 0).all()
        check(r, cache, q, cu, ln, table, 0.125, rows=slice(new, None))


@pytest.mark.parametrize("news,most", [([3, 1], 2), ([200, 90], 100)])
def test_a_sequence_of_more_rows_than_said_is_left_out(news, most):
    cache, ln, table = filled("nvfp4", [300, 300], 1, 16, 128, 3)
    cu = dev32([0, news[0], sum(news)])
    q = torch.randn((sum(news), 4, 128), generator=gen(1), device="cuda").bfloat16()
    r = mxq.cache_attention(cache, q, cu, ln, table, most)
    assert r["status"].item() == mxq.DEV_INVALID_PAGE and (r["o"][:news[0]] == 0).all()
    check(r, cache, q, cu, ln, table, 128 ** -0.5, rows=slice(news[0], None))


def test_batches_that_are_not_in_order_touch_nothing_else():
    """cu that descends or leaves the tensor: no row of such a sequence is read or written."""
    cache, ln, table = filled("mxfp8", [50, 50, 50], 1, 16, 64, 3)
    q = torch.randn((6, 2, 64), generator=gen(1), device="cuda").bfloat16()
    for cu, good in (([0, 4, 2, 6], [0, 1, 2, 3]), ([-3, 2, 4, 6], [2, 3, 4, 5]), ([0, 2, 4, 9], [0, 1, 2, 3])):
        r = mxq.cache_attention(cache, q, dev32(cu), ln, table, 4)
        for row in range(6):
            if row not in good and not (cu[2] == 2 and row in (2, 3, 4, 5)):
                assert (r["o"][row] == 0).all()


def test_empty_batches():
    cache, ln, table = filled("mxfp8", [50], 1, 16, 64, 3)
    q = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert mxq.cache_attention(cache, q, dev32([0, 0]), ln, table, 0)["o"].shape == (0, 2, 64)
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    for most in (0, 1, 200):
        r = mxq.cache_attention(cache, q, dev32([1, 1]), ln, table, most)
        assert (r["o"] == 0).all() and r["status"].item() == 0
    r = mxq.cache_attention(cache, q, dev32([0]), dev32([]), table[:0], 1)
    assert (r["o"] == 0).all()


@pytest.mark.parametrize("new", [1, 64])
def test_codes_behind_the_fourth_gibibyte(new):
    """Pages 17000 and on of 256 KB: byte offsets past 32 bits."""
    cache = mxq.Cache.empty(1, 4, 256, 256, "mxfp8")
    shape = lambda w: (17100, 4, 256, w)  # noqa: E731
    cache = mxq.Cache(*(torch.empty(shape(w), dtype=torch.uint8, device="cuda") for w in (256, 8, 256, 8)))
    ln, table = dev32([700]), dev32([[17098, 16999, 17005]])
    k, v = (torch.randn((700, 4, 256), generator=gen(i), device="cuda").bfloat16() for i in range(2))
    mxq.cache_write(cache, k, v, dev32([0, 700]), ln, table)
    back = mxq.cache_read(cache, dev32([0, 700]), ln, table, 700)
    assert (back["k"].float() - k.float()).abs().max() < 0.5
    q = torch.randn((new, 8, 256), generator=gen(4), device="cuda").bfloat16()
    cu = dev32([0, new])
    check(mxq.cache_attention(cache, q, cu, ln, table, new), cache, q, cu, ln, table, 1 / 16)


def test_pages_that_sequences_share():
    """A common beginning on the same pages."""
    cache, ln, table = filled("nvfp4", [64, 90], 2, 16, 128, 3)
    table[1, :4] = table[0, :4]
    q = torch.randn((2, 8, 128), generator=gen(4), device="cuda").bfloat16()
    cu = dev32([0, 1, 2])
    check(mxq.cache_attention(cache, q, cu, ln, table, 1), cache, q, cu, ln, table, 128 ** -0.5)


@pytest.mark.parametrize("new", [1, 70])
def test_captured_replayed_and_side_by_side(new):
    """Two calls in one graph on two streams, each with its own workspace; replays see new
    queries and a longer sequence."""
    cache, ln, table = filled("mxfp8", [3000, 500], 2, 64, 128, 3)
    q = torch.randn((2 * new, 8, 128), generator=gen(4), device="cuda").bfloat16()
    cu = dev32([0, new, 2 * new])
    ws = [mxq.cache_attention_workspace(cache, 2 * new, 8, 2, new) for _ in range(2)]
    o = [torch.empty((2 * new, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def go(i, scale, stream=None):
        mxq.mxq_cache_attention(cache, q, 1024, 2 * new, 8, cu, ln, table, 2, table.shape[1], new, scale, o[i], None, st, ws[i], stream)
    go(0, 0.1), go(1, 0.2)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        go(0, 0.1)
        go(1, 0.2, side)
        torch.cuda.current_stream().wait_stream(side)
    for seed, n in ((5, 2000), (6, 3000)):
        q.copy_(torch.randn(q.shape, generator=gen(seed), device="cuda"))
        ln[0] = n
        graph.replay()
        for i, scale in enumerate((0.1, 0.2)):
            assert torch.equal(o[i], mxq.cache_attention(cache, q, cu, ln, table, new, scale=scale)["o"])


def test_host_threads_with_streams_of_their_own():
    """Calls of different sizes from several threads at once, against the same calls one by one."""
    work = []
    for seed, (lens, new, group, dim, fmt) in enumerate((([3000, 70], 1, 8, 128, "mxfp8"), ([900], 300, 2, 64, "nvfp4"),
                                                         ([40] * 9, 4, 3, 256, "nvfp4"), ([2000, 10], 33, 4, 256, "mxfp8"))):
        cache, ln, table = filled(fmt, lens, 2, 16, dim, seed)
        q = torch.randn((new * len(lens), 2 * group, dim), generator=gen(seed), device="cuda").bfloat16()
        w = layers.quantize_projection(torch.randn((700, 256), generator=gen(seed), device="cuda").bfloat16(), fmt)
        x = torch.randn((new, 256), generator=gen(seed), device="cuda").bfloat16()
        cu = dev32([i * new for i in range(len(lens) + 1)])
        work.append(lambda stream, c=(cache, q, cu, ln, table, new), x=x, w=w, fmt=fmt: (
            mxq.cache_attention(*c, stream=stream)["o"], mxq.linear(x, w, fmt, stream=stream)["y"]))
    want = [f(None) for f in work]
    torch.cuda.synchronize()
    got, failed = [[None] * 20 for _ in work], []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            for n in range(20):
                got[i][n] = work[i](stream)
            stream.synchronize()
        except Exception as e:
            failed.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for a, b in zip(got, want):
        for o, y in a:
            assert torch.equal(o, b[0]) and torch.equal(y, b[1])


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_a_sequence_from_its_prompt_through_decoding(fmt):
    """The operators as a model uses them: projections over a quantized matrix, the new tokens
    written and attended to, in chunks and then one by one, against binary64 over what the
    cache holds at each step."""
    H, heads, kv, dim, tokens = 256, 8, 2, 64, 32
    w_qkv = layers.quantize_projection(torch.randn(((heads + 2 * kv) * dim, H), generator=gen(1), device="cuda").bfloat16() * 0.06, "nvfp4")
    w_out = layers.quantize_projection(torch.randn((H, heads * dim), generator=gen(2), device="cuda").bfloat16() * 0.05, "mxfp8")
    s2 = (torch.full((kv,), 0.002, device="cuda"),) * 2 if fmt == "nvfp4" else (None, None)
    cache = mxq.Cache.empty(20, kv, tokens, dim, fmt, *s2)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1))[:16].view(2, 8).int().cuda()
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for step, news in enumerate(([100, 37], [60, 1], [1, 1], [1, 3], [1, 0], [1, 1])):
        T = sum(news)
        cu = dev32([0, news[0], T])
        lens += dev32(news)
        x = torch.randn((T, H), generator=gen(10 + step), device="cuda").bfloat16()
        qkv = layers.projection_forward(w_qkv, x)["y"].view(T, heads + 2 * kv, dim)
        r = layers.attention_forward(cache, qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:], cu, lens, table, max(news))
        assert r["status"].item() == 0
        check(r, cache, qkv[:, :heads], cu, lens, table, dim ** -0.5)
        y = layers.projection_forward(w_out, r["o"].view(T, heads * dim), out="f32")["y"].double()
        d = ref.values(w_out["codes"], w_out["scales"], "mxfp8")
        a = r["o"].view(T, -1).double()
        assert ((y - a @ d.t()).abs() <= a.abs() @ d.t().abs() * 2.0 ** -16 + 1e-30).all()
    # the whole sequences back
    whole = mxq.cache_read(cache, dev32([0, int(lens[0]), int(lens.sum())]), lens, table, int(lens.sum()))
    k0 = ref.sequence_values(cache, 0, lens, table)[0]
    assert ((whole["k"][:int(lens[0])].double() - k0).abs() <= k0.abs() * 2.0 ** -8).all()

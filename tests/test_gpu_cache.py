"""The quantized key/value cache on the GPU: what is written, bit for bit, where it is
written, and what is read back."""
import pytest
import torch

import cache_ref as ref
from mxfp_block_scaled_b200 import mxq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def dev32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make_cache(fmt, pages, heads, tokens, dim, seed=0, fill=0xA5):
    s2 = (None, None)
    if fmt == "nvfp4":
        s2 = tuple(torch.exp2(torch.rand(heads, generator=gen(seed + i), device="cuda") * 6 - 10) for i in range(2))
    c = mxq.Cache.empty(pages, heads, tokens, dim, fmt, *s2)
    for t in c.tensors[:4]:
        t.fill_(fill)
    return c


def batch(news, lens, tokens, pages, seed, first=0):
    """cu, lens and a table of distinct pages in a shuffled order."""
    width = max(-(-max(lens + [1]) // tokens), 1)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(news), width), -7, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // tokens)):
            table[b, i] = order.pop()
    cu = [first]
    for n in news:
        cu.append(cu[-1] + n)
    return dev32(cu), dev32(lens), table.cuda()


def expect(cache, x, s2, mode):
    """(codes, scales) of rows x [T, heads, dim] as the tensor quantizers give them."""
    T, H, D = x.shape
    if cache.fmt == "mxfp8":
        q = mxq.quantize_mx(x.reshape(T * H, D).contiguous(), "mxfp8")
        return q["codes"].view(T, H, D), q["scales"].view(T, H, -1)
    q = mxq.quantize_nvfp4_s2(x.transpose(0, 1).contiguous(), s2, mode=mode)
    return q["codes"].transpose(0, 1), q["scales"].transpose(0, 1)


@pytest.mark.parametrize("fmt,mode", [("mxfp8", "rtn"), ("nvfp4", "rtn"), ("nvfp4", "four_six")])
@pytest.mark.parametrize("news,lens,heads,tokens,dim,strided", [
    ([1], [1], 1, 16, 64, False), ([1, 1, 1], [17, 1, 300], 2, 16, 128, True), ([5, 0, 700, 1], [5, 40, 1000, 257], 3, 64, 64, True),
    ([33], [33], 5, 256, 256, False), ([130, 7], [400, 7], 8, 32, 128, True), ([2] * 70, list(range(2, 72)), 1, 16, 64, False),
    ([3, 2000], [9, 2100], 40, 128, 64, False)])
def test_writes_what_the_quantizers_give_and_nothing_else(fmt, mode, news, lens, heads, tokens, dim, strided):
    first, pad = 2, 3
    T = first + sum(news) + pad
    pages = sum(-(-n // tokens) for n in lens) + 2
    cache = make_cache(fmt, pages, heads, tokens, dim)
    cu, ln, table = batch(news, lens, tokens, pages, 1, first)
    wide = torch.randn((T, 2 * heads + 1, dim), generator=gen(T), device="cuda").bfloat16()
    wide *= torch.exp2(torch.randint(-8, 9, (T, 2 * heads + 1, 1), generator=gen(3), device="cuda").float()).bfloat16()
    k, v = wide[:, 1:1 + heads], wide[:, 1 + heads:]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    want = [t.clone() for t in cache.tensors[:4]]
    rows, _, _, page, tok = (torch.tensor(c, device="cuda") for c in zip(*ref.places(cu, ln, table, tokens, pages)))
    for i, (x, s2) in enumerate(((k, cache.k_s2), (v, cache.v_s2))):
        codes, scales = expect(cache, x, s2, mode)
        want[2 * i][page, :, tok], want[2 * i + 1][page, :, tok] = codes[rows], scales[rows]
    st = mxq.cache_write(cache, k, v, cu, ln, table, mode=mode)
    assert st.item() == 0
    for got, w in zip(cache.tensors[:4], want):
        assert torch.equal(got, w)
    # and back: every row of a sequence, the others left as they were
    out = {n: torch.full((T, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda") for n in "kv"}
    mxq.mxq_cache_read(cache, cu, ln, table, len(news), table.shape[1], T, out["k"], out["v"], st)
    for n, codes, scales, s2 in (("k", want[0], want[1], cache.k_s2), ("v", want[2], want[3], cache.v_s2)):
        if fmt == "mxfp8":
            x = ref.values(codes[page, :, tok], scales[page, :, tok], fmt).to(torch.bfloat16)
        else:
            x = ref.values(codes[page, :, tok], scales[page, :, tok], fmt, torch.ones_like(s2)[None].expand(len(rows), -1))
            x = (x.float() * s2[None, :, None]).to(torch.bfloat16)
        y = torch.full_like(out[n], 9.0)
        y[rows] = x
        assert torch.equal(out[n].view(torch.int16), y.view(torch.int16))
    assert st.item() == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_rows_without_a_place_and_bad_pages(fmt):
    """Sequence 0 has fewer tokens than rows, 1 a page that is none, 2 ends behind the table, 3 is
    in order, 4 has no token at all."""
    cache = make_cache(fmt, 6, 2, 16, 64)
    news, lens = [5, 20, 10, 4, 2], [3, 40, 40, 8, 0]
    cu, ln = dev32([0, 5, 25, 35, 39, 41]), dev32(lens)
    table = dev32([[0, -1], [1, 6], [2, 3], [4, 1 << 30], [-5, -5]])
    T = 41
    k, v = (torch.randn((T, 2, 64), generator=gen(i), device="cuda").bfloat16() for i in range(2))
    want = [t.clone() for t in cache.tensors[:4]]
    rows, _, _, page, tok = (torch.tensor(c, device="cuda") for c in zip(*ref.places(cu, ln, table, 16, 6)))
    for i, (x, s2) in enumerate(((k, cache.k_s2), (v, cache.v_s2))):
        codes, scales = expect(cache, x, s2, "rtn")
        want[2 * i][page, :, tok], want[2 * i + 1][page, :, tok] = codes[rows], scales[rows]
    st = mxq.cache_write(cache, k, v, cu, ln, table)
    assert st.item() == mxq.DEV_INVALID_PAGE
    for got, w in zip(cache.tensors[:4], want):
        assert torch.equal(got, w)
    out = mxq.cache_read(cache, cu, ln, table, T)
    assert out["status"].item() == mxq.DEV_INVALID_PAGE
    lost = torch.ones(T, dtype=torch.bool, device="cuda")
    lost[rows] = False
    assert (out["k"][lost] == 0).all() and (out["k"][rows].float() - k[rows].float()).abs().max() < 1
    # the sequence in order alone sets nothing
    st = mxq.cache_write(cache, k[35:39], v[35:39], dev32([0, 4]), ln[3:4], table[3:4])
    assert st.item() == 0


def test_nonfinite_values_and_scales_are_reported():
    x = torch.randn((4, 2, 64), generator=gen(1), device="cuda").bfloat16()
    cu, ln, table = dev32([0, 4]), dev32([4]), dev32([[1]])
    for fmt in ("mxfp8", "nvfp4"):
        for bad in (float("inf"), float("-inf"), float("nan")):
            cache, y = make_cache(fmt, 2, 2, 16, 64), x.clone()
            y[2, 1, 63] = bad
            assert mxq.cache_write(cache, x, y, cu, ln, table).item() == mxq.DEV_NONFINITE_INPUT
            good = make_cache(fmt, 2, 2, 16, 64)
            mxq.cache_write(good, x, x, cu, ln, table)
            assert torch.equal(cache.k_codes, good.k_codes)
            assert torch.equal(cache.v_codes[:, 0], good.v_codes[:, 0])
            # of rows that have no place nothing is said
            st = mxq.cache_write(cache, x, y, dev32([0, 2]), dev32([2]), table)
            assert st.item() == 0
    for s2 in (-1.0, float("inf"), float("nan")):
        cache = make_cache("nvfp4", 2, 2, 16, 64)
        cache.v_s2[1] = s2
        assert mxq.cache_write(cache, x, x, cu, ln, table).item() == mxq.DEV_INVALID_SCALE
        assert (cache.v_codes[:, 1] == 0xA5).all() and not (cache.v_codes[1, 0, :4] == 0xA5).all()
    cache = make_cache("nvfp4", 2, 2, 16, 64)       # a scale of zero: a head of zeros
    cache.v_s2[1] = 0.0
    assert mxq.cache_write(cache, x, x, cu, ln, table).item() == 0
    assert (cache.v_codes[1, 1, :4] == 0).all() and (cache.v_scales[1, 1, :4] == 0).all()
    assert (mxq.cache_read(cache, cu, ln, table, 4)["v"][:, 1] == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_zeros_a_captured_write_and_an_empty_batch(fmt):
    cache = make_cache(fmt, 3, 2, 32, 128)
    x = torch.zeros((6, 2, 128), dtype=torch.bfloat16, device="cuda")
    cu, ln, table = dev32([0, 6]), dev32([6]), dev32([[2]])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mxq.cache_write(cache, x, x, cu, ln, table, status=st)
    assert (mxq.cache_read(cache, cu, ln, table, 6)["k"] == 0).all()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mxq.mxq_cache_write(cache, x, 256, x, 256, 6, cu, ln, table, 1, 1, "rtn", st)
    for n in (6, 20):           # a later length moves the rows
        x.copy_(torch.randn(x.shape, generator=gen(n), device="cuda"))
        ln.fill_(n)
        graph.replay()
        got = mxq.cache_read(cache, cu, ln, table, 6)["v"].float()
        assert ((got - x.float()).abs() <= x.float().abs().amax(-1, keepdim=True) / 3).all()
    before = [t.clone() for t in cache.tensors[:4]]
    none = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    mxq.cache_write(cache, none, none, dev32([0, 0]), dev32([9]), table, status=st)
    mxq.cache_write(cache, none, none, dev32([0]), dev32([]), table[:0], status=st)
    assert mxq.cache_read(cache, dev32([0, 0]), dev32([9]), table, 0)["k"].shape == (0, 2, 128)
    assert all(torch.equal(a, b) for a, b in zip(before, cache.tensors[:4])) and st.item() == 0

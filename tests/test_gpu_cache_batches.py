"""Batches whose rows are not the call's: what each call on a cache leaves out, what it does
for the others, and that all of them say so."""
import pytest
import torch

from mxfp_block_scaled_b200 import mxq
from test_gpu_cache import dev32, gen, make_cache
from test_gpu_cache_attention import filled

pytestmark = pytest.mark.gpu
# cu, and the sequences that are in order with their rows
BAD = [([4, 2, 4, 6], {1: (2, 4), 2: (4, 6)}), ([-3, 2, 4, 6], {1: (2, 4), 2: (4, 6)}), ([0, 2, 4, 9], {0: (0, 2), 1: (2, 4)}),
       ([0, 2, 1, 6], {0: (0, 2), 2: (1, 6)}), ([-5, -2, 3, 3], {2: (3, 3)}), ([0, 3, 2 ** 31 - 1, -2 ** 31], {0: (0, 3)}),
       ([7, 9, 11, 12], {})]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


@pytest.mark.parametrize("group", [2, 40])
@pytest.mark.parametrize("cu,good", BAD)
def test_attention_leaves_them_out(cu, good, group):
    cache, ln, table = filled("mxfp8", [50, 50, 50], 1, 16, 64, 3)
    q = torch.randn((6, group, 64), generator=gen(1), device="cuda").bfloat16()
    r = mxq.cache_attention(cache, q, dev32(cu), ln, table, 6)
    assert r["status"].item() == mxq.DEV_INVALID_PAGE
    rows = [row for r0, r1 in good.values() for row in range(r0, r1)]
    for b, (r0, r1) in good.items():
        want = mxq.cache_attention(cache, q[:r1], dev32([r0, r1]), ln[b:b + 1], table[b:b + 1], 6)
        assert want["status"].item() == 0
        for row in range(r0, r1):
            if rows.count(row) == 1:        # (of a row that two sequences claim the result is either's)
                # both are within 2^-8 of the result and 2^-11 of sum p |v|, which is below 16
                x, y = r["o"][row].float(), want["o"][row].float()
                assert ((x - y).abs() <= 2.0 ** -7 * torch.maximum(x.abs(), y.abs()) + 2.0 ** -6).all()
    rest = [row for row in range(6) if row not in rows]
    assert (r["o"][rest] == 0).all() and (r["lse"][rest] == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("cu,good", BAD)
def test_write_and_read_leave_them_out(cu, good, fmt):
    cache = make_cache(fmt, 4, 2, 16, 64)
    ln, table = dev32([9, 9, 9]), dev32([[0], [2], [3]])
    x = torch.randn((6, 2, 64), generator=gen(1), device="cuda").bfloat16()
    before = [t.clone() for t in cache.tensors[:4]]
    assert mxq.cache_write(cache, x, x, dev32(cu), ln, table).item() == mxq.DEV_INVALID_PAGE
    out = mxq.cache_read(cache, dev32(cu), ln, table, 6)
    assert out["status"].item() == mxq.DEV_INVALID_PAGE
    ascending = all(b >= a for a, b in zip(cu, cu[1:]))
    want, may = make_cache(fmt, 4, 2, 16, 64), torch.zeros(6, dtype=torch.bool, device="cuda")
    for b, (r0, r1) in good.items():
        may[r0:r1] = True
        if r1 > r0:
            assert mxq.cache_write(want, x[:r1], x[:r1], dev32([r0, r1]), ln[b:b + 1], table[b:b + 1]).item() == 0
    for got, w, old in zip(cache.tensors[:4], want.tensors[:4], before):
        assert ((got == w) | (got == old)).all() and (torch.equal(got, w) or not ascending)
    assert (out["k"][~may] == 0).all()
    if ascending:
        assert (out["k"][may] != 0).any(-1).all()


def test_batches_in_order_say_nothing():
    """Empty sequences, rows before the first and behind the last, all rows of the call."""
    cache, ln, table = filled("mxfp8", [50, 50, 50], 1, 16, 64, 3)
    x = torch.randn((6, 1, 64), generator=gen(1), device="cuda").bfloat16()
    for cu in ([0, 2, 4, 6], [1, 1, 1, 5], [0, 0, 6, 6], [6, 6, 6, 6], [0, 0, 0, 0]):
        assert mxq.cache_write(cache, x, x, dev32(cu), ln, table).item() == 0
        assert mxq.cache_read(cache, dev32(cu), ln, table, 6)["status"].item() == 0
        assert mxq.cache_attention(cache, x.expand(6, 1, 64), dev32(cu), ln, table, 6)["status"].item() == 0

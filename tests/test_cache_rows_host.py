"""Rows of the calls on a cache as the binding takes them, without a GPU (the compute entry
points are replaced by a recorder; host tensors stand in for device tensors): bf16 values, each
row's contiguous, the rows as far apart as the call says."""
import pytest
import torch

from mxfp_block_scaled_b200 import mxq
from test_cache_ops_host import a_batch, a_cache, bf16, i32, lib, rec, u8  # noqa: F401


def calls(k, q, ks=128, qs=256, T=4):
    cache, b, st = a_cache(), a_batch(), i32(0)
    return [lambda: mxq.mxq_cache_write(cache, k, ks, bf16(4, 128), 128, T, *b, 2, 2, "rtn", st),
            lambda: mxq.mxq_cache_write(cache, bf16(4, 128), 128, k, ks, T, *b, 2, 2, "rtn", st),
            lambda: mxq.mxq_cache_attention(cache, q, qs, T, 4, *b, 2, 2, 2, 1.0, bf16(4, 256), None, st, u8(1 << 20))]


def test_contiguous_rows_and_columns_of_wider_ones_are_taken(rec):  # noqa: F811
    wide = bf16(4, 10, 64)
    for go in calls(bf16(4, 2, 64), bf16(4, 4, 64)) + calls(bf16(4, 128), bf16(1024)) + calls(wide[:, 3:5], wide[:, 5:9], 640, 640) \
            + calls(bf16(1, 2, 64).expand(1, 2, 64), bf16(1, 4, 64), T=1) + calls(bf16(4, 1, 2, 64), bf16(4, 2, 2, 64)):
        go()
    assert len(rec.calls) == 15


@pytest.mark.parametrize("k,q", [
    (torch.zeros(4, 2, 64), torch.zeros(4, 4, 64)), (torch.zeros(4, 2, 64).half(), torch.zeros(4, 4, 64).half()),
    (u8(4, 512), u8(4, 1024))])
def test_other_types_are_refused(rec, k, q):  # noqa: F811
    for go in calls(k, q):
        with pytest.raises(ValueError, match="bf16"):
            go()
    assert not rec.calls


@pytest.mark.parametrize("k,q,ks,qs", [
    (bf16(4, 2, 128)[..., ::2], bf16(4, 4, 128)[..., ::2], 256, 512),                       # every second value
    (bf16(4, 64, 2).transpose(1, 2), bf16(4, 64, 4).transpose(1, 2), 128, 256),
    (bf16(4, 4, 64)[:, ::2], bf16(4, 8, 64)[:, ::2], 256, 512),                             # every second head
    (bf16(4, 2, 64), bf16(4, 4, 64), 136, 264), (bf16(4, 3, 64)[:, :2], bf16(4, 5, 64)[:, :4], 128, 256)])   # another stride than said
def test_rows_that_lie_otherwise_are_refused(rec, k, q, ks, qs):  # noqa: F811
    for go in calls(k, q, ks, qs):
        with pytest.raises(ValueError):
            go()
    assert not rec.calls

"""Attention's waits that run out, on the GPU without faulting or hanging it: a launch told to
stall (include/mxq_test.h: keys or values of one step are never reported as there) must end on
its own with MXQ_DEV_WAIT_TIMEOUT and write nothing beside its results, and the next calls must
give the bits of the calls before.  The failure is made by the host-side request; no trap,
assert or bad address is involved."""
import time

import pytest
import torch

from mxfp_block_scaled_b200 import mxq
from test_gpu_cache import dev32, gen
from test_gpu_cache_attention import filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def case(fmt, dim, new, group, length):
    cache, ln, table = filled(fmt, [length], 4, 32, dim, 3)
    q = torch.randn((new, 4 * group, dim), generator=gen(1), device="cuda").bfloat16()
    return cache, q, dev32([0, new]), ln, table, new


# tiles of two groups, of one (64 rows, and heads of 256), and a CTA's way from one tile to the next
CASES = [("mxfp8", 128, 600, 16, 4000), ("nvfp4", 64, 70, 1, 20000), ("mxfp8", 256, 300, 8, 3000), ("nvfp4", 128, 3000, 2, 3000)]


@pytest.mark.parametrize("step", [0, 1, 7])
@pytest.mark.parametrize("what", ["keys", "values"])
@pytest.mark.parametrize("fmt,dim,new,group,length", CASES)
def test_stalled_attention_reports_wait_timeout_and_the_device_recovers(fmt, dim, new, group, length, what, step):
    c = case(fmt, dim, new, group, length)
    want = mxq.cache_attention(*c)
    assert want["status"].item() == 0
    cache, q, cu, ln, table, _ = c
    n, pad = q.numel(), 4096
    full = torch.full((n + 2 * pad,), 5.0, device="cuda", dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = mxq.cache_attention_workspace(cache, new, q.shape[1], 1, new)
    ws.zero_()
    lib = mxq.load()
    torch.cuda.synchronize()
    lib.mxq_test_stall_next_attention((1 if what == "keys" else 2) + 2 * step)
    t0 = time.perf_counter()
    mxq.mxq_cache_attention(cache, q, q.stride(0), new, q.shape[1], cu, ln, table, 1, table.shape[1], new, 0.1,
                            full[pad:pad + n], None, st, ws)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert int(st.item()) == mxq.DEV_WAIT_TIMEOUT
    assert elapsed < 5.0, elapsed
    assert bool((full[:pad] == 5).all()) and bool((full[pad + n:] == 5).all())
    for _ in range(3):
        r = mxq.cache_attention(*c, workspace=ws)
        assert r["status"].item() == 0 and torch.equal(r["o"], want["o"]) and torch.equal(r["lse"], want["lse"])


def test_stalled_attention_between_others():
    """Launches before and after a stalled one, queued without waiting for it, are ordinary."""
    c = case("mxfp8", 128, 300, 8, 2000)
    want, lib, outs = mxq.cache_attention(*c), mxq.load(), []
    torch.cuda.synchronize()
    for i in range(6):
        lib.mxq_test_stall_next_attention(4 if i == 2 else 0)
        outs.append(mxq.cache_attention(*c))
    torch.cuda.synchronize()
    for i, r in enumerate(outs):
        assert int(r["status"].item()) == (mxq.DEV_WAIT_TIMEOUT if i == 2 else 0)
        assert i == 2 or torch.equal(r["o"], want["o"])


def test_withdrawn_and_ignored_stall_requests_change_nothing():
    c, lib = case("mxfp8", 128, 100, 4, 500), mxq.load()
    want = mxq.cache_attention(*c)["o"]
    lib.mxq_test_stall_next_attention(1)
    lib.mxq_test_stall_next_attention(0)
    r = mxq.cache_attention(*c)
    assert r["status"].item() == 0 and torch.equal(r["o"], want)
    lib.mxq_test_stall_next_attention(1)
    assert mxq.cache_attention(*case("mxfp8", 128, 1, 4, 500))["status"].item() == 0       # few rows: no waits
    lib.mxq_test_stall_next_attention(0)

"""The block-FP8 product's waits that run out, on the GPU without faulting or
hanging it: a launch told to stall (include/mxq_test.h: the scales of one step
are never reported as there) must end on its own with MXQ_DEV_WAIT_TIMEOUT and
write nothing beside its result, and the next calls must give the bits of the
calls before.  The failure is made by the host-side request; no trap, assert or
bad address is involved."""
import time

import pytest
import torch

from mxfp_block_scaled_b200 import mxq, workloads

pytestmark = pytest.mark.gpu

# tiles of 64, 128 and 256 columns, some items a CTA; tiles shared by clusters of two and of four
SIZES = [(1100, 64, 272), (2500, 520, 400), (4096, 2560, 2048), (700, 310, 16), (129, 640, 2192), (64, 1536, 2048), (64, 512, 8192)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def _operands(M, N, K):
    a = mxq.quantize_fp8(workloads.activation_tile(M, seed=M, device="cuda", hidden=K))
    w = torch.randn((N, K), generator=torch.Generator(device="cuda").manual_seed(N), device="cuda") * 0.02
    b = mxq.quantize_fp8(w.to(torch.bfloat16), brows=128)
    return a["codes"], a["scales"], b["codes"], b["scales"]


@pytest.mark.parametrize("step", [1, 2])      # the first step's wait runs out, the last one's
@pytest.mark.parametrize("M,N,K", SIZES)
def test_stalled_product_reports_wait_timeout_and_the_device_recovers(M, N, K, step):
    ops = _operands(M, N, K)
    want = mxq.gemm_fp8(*ops, out="f32")["c"]
    pad = 4096
    full = torch.full((M * N + 2 * pad,), 5.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib = mxq.load()
    torch.cuda.synchronize()
    lib.mxq_test_stall_next_product(step)
    t0 = time.perf_counter()
    mxq.mxq_gemm_fp8(*ops, M, N, K, "f32", full[pad:pad + M * N], st)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert int(st.item()) == mxq.DEV_WAIT_TIMEOUT
    assert elapsed < 5.0, elapsed
    assert bool((full[:pad] == 5).all()) and bool((full[pad + M * N:] == 5).all())
    # the request was taken by that launch; the next ones are ordinary
    for _ in range(5):
        r = mxq.gemm_fp8(*ops, out="f32")
        assert int(r["status"].item()) == 0 and torch.equal(r["c"], want)


def test_stalled_product_between_others():
    """Launches before and after a stalled one, queued without waiting for it, are ordinary."""
    ops = _operands(500, 700, 1040)
    want = mxq.gemm_fp8(*ops)["c"]
    lib = mxq.load()
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        lib.mxq_test_stall_next_product(1 if i == 2 else 0)
        outs.append(mxq.gemm_fp8(*ops))
    torch.cuda.synchronize()
    for i, r in enumerate(outs):
        assert int(r["status"].item()) == (mxq.DEV_WAIT_TIMEOUT if i == 2 else 0)
        assert i == 2 or torch.equal(r["c"], want)


def test_withdrawn_and_ignored_stall_requests_change_nothing():
    lib, ops = mxq.load(), _operands(300, 400, 640)
    want = mxq.gemm_fp8(*ops)["c"]
    lib.mxq_test_stall_next_product(1)
    lib.mxq_test_stall_next_product(0)
    r = mxq.gemm_fp8(*ops)
    assert int(r["status"].item()) == 0 and torch.equal(r["c"], want)
    few = _operands(4, 400, 640)
    lib.mxq_test_stall_next_product(2)                      # streamed: no waits
    assert int(mxq.gemm_fp8(*few)["status"].item()) == 0
    lib.mxq_test_stall_next_product(0)

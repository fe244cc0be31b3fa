"""Block-FP8 quantizer on the GPU against its definition: codes and scales bit
for bit."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from mxfp_block_scaled_b200 import mxq, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def _check_quant(x, brows, guard=256):
    """Quantize x [R, C] (bf16, on the GPU) into guarded buffers and compare."""
    R, C = x.shape
    ns = -(-R // brows) * -(-C // 128)
    codes = torch.full((R * C + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((ns + 2 * guard,), -7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mxq.mxq_quantize_fp8(x, R, C, brows, 128, codes[guard:guard + R * C], scales[guard:guard + ns], st)
    c, s = ref.quantize_fp8(x.float().cpu().numpy(), brows)
    assert int(st.item()) == 0
    assert np.array_equal(scales[guard:guard + ns].cpu().numpy().view(np.uint32), s.ravel().view(np.uint32))
    assert np.array_equal(codes[guard:guard + R * C].cpu().numpy(), c.ravel())
    for buf, n, fill in ((codes, R * C, 0xA5), (scales, ns, -7.0)):
        assert bool((buf[:guard] == fill).all()) and bool((buf[guard + n:] == fill).all())


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 2048), (2, 128), (3, 144), (17, 1552), (129, 272), (128, 128),
                                       (300, 2048), (5000, 176), (1, 16384), (2500, 2048)])
@pytest.mark.parametrize("brows", [1, 128])
def test_quantize_bit_exact(rows, cols, brows):
    _check_quant(workloads.activation_tile(rows, seed=rows + cols, device="cuda", hidden=cols), brows)


@pytest.mark.parametrize("brows", [1, 128])
def test_quantize_ranges(brows):
    """Blocks of zeros (with -0), of the smallest and largest bf16 magnitudes, mixed
    signs, values at and around the rounding ties, and scales past both ends of
    the reciprocal's range."""
    g = torch.Generator().manual_seed(5)
    rows = []
    for e in (-133, -130, -126, -118, -117, -70, -60, -52, -51, -50, -1, 0, 40, 60, 68, 69, 70, 100, 119, 127):
        m = torch.randint(128, 256, (128,), generator=g).float() / 128
        drop = torch.randint(0, 24, (128,), generator=g).float()
        v = torch.ldexp(m.double(), (e - drop).double()) * (torch.randint(0, 2, (128,), generator=g) * 2 - 1)
        v[0] = 2.0 ** e
        rows.append(v.to(torch.bfloat16))
    rows.append(torch.zeros(128, dtype=torch.bfloat16))
    rows.append(-torch.zeros(128, dtype=torch.bfloat16))
    ties = torch.tensor([448.0] + [(ref.GRID[i] + ref.GRID[i + 1]) / 2 for i in range(126)] + [-0.0])
    rows.append(ties.to(torch.bfloat16))              # scale 1: the quotient is the value
    x = torch.stack(rows).cuda()
    if brows == 128:                                  # each row a block of its own: 128 equal rows
        x = x.repeat_interleave(128, 0)
    _check_quant(x.contiguous(), brows)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("brows", [1, 128])
def test_quantize_nonfinite_sets_status(bad, brows):
    x = workloads.activation_tile(130, seed=3, device="cuda", hidden=272)
    assert int(mxq.quantize_fp8(x, brows)["status"].item()) == 0
    x[129, 271] = bad
    assert int(mxq.quantize_fp8(x, brows)["status"].item()) == mxq.DEV_NONFINITE_INPUT


def test_codes_feed_the_requantizer():
    """The quantizer's output is the requantizer's input format, for both block shapes."""
    import oracle
    oracle.build()
    x = workloads.activation_tile(200, seed=8, device="cuda", hidden=384)
    for brows in (1, 128):
        q = mxq.quantize_fp8(x, brows)
        out = mxq.requant_fp8_mx(q["codes"], q["scales"], brows, 128, "mxfp8")
        oc, os_ = oracle.requant_fp8_mx(q["codes"].cpu().numpy(), q["scales"].cpu().numpy(), brows, 128, "mxfp8")
        assert np.array_equal(out["codes"].cpu().numpy(), oc) and np.array_equal(out["scales"].cpu().numpy(), os_)


def test_large_tile_by_rows():
    """A tile whose codes pass 2^31 bytes: the last rows equal those rows quantized alone."""
    rows, cols = 140000, 16384
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16).random_(0, 0x4200)            # positive finite values
    q = mxq.quantize_fp8(x)
    part = mxq.quantize_fp8(x[-128:].contiguous())
    assert torch.equal(q["codes"][-128:], part["codes"]) and torch.equal(q["scales"][-128:], part["scales"])
    w = mxq.quantize_fp8(x, brows=128)
    part = mxq.quantize_fp8(x[128 * 1093:].contiguous(), brows=128)
    assert torch.equal(w["codes"][128 * 1093:], part["codes"]) and torch.equal(w["scales"][1093:], part["scales"])


@pytest.mark.parametrize("rows,cols", [(4097, 2048), (4201, 2000), (66001, 16), (40000, 144)])
def test_quantize_many_blocks_bit_exact(rows, cols):
    _check_quant(workloads.activation_tile(rows, seed=cols, device="cuda", hidden=cols), 1)

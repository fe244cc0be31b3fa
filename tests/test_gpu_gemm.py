"""Block-FP8 matrix product on the GPU against its definition in binary64,
elementwise inside a bound derived from the roundings (layer_ref)."""
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


def operands(M, N, K, seed=0):
    a = mxq.quantize_fp8(workloads.activation_tile(M, seed=seed, device="cuda", hidden=K))
    w = (torch.randn((N, K), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * 0.02)
    b = mxq.quantize_fp8(w.to(torch.bfloat16), brows=128)
    return a["codes"], a["scales"], b["codes"], b["scales"]


def check(ops, out, pad=512):
    """Into a guarded buffer; compared elementwise."""
    M, N, K = ops[0].shape[0], ops[2].shape[0], ops[0].shape[1]
    full = torch.full((M * N + 2 * pad,), 7.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    c, st = full[pad:pad + M * N], torch.zeros(1, dtype=torch.int32, device="cuda")
    mxq.mxq_gemm_fp8(*ops, M, N, K, out, c, st)
    assert int(st.item()) == 0
    assert bool((full[:pad] == 7).all()) and bool((full[pad + M * N:] == 7).all())
    want, bound = ref.gemm(*(t.cpu().numpy() for t in ops), out)
    ref.close(c.view(M, N), want, bound)
    return c.view(M, N)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 2560, 2048), (3, 17, 48), (8, 129, 128), (9, 100, 272), (16, 2048, 1280),
                                   (17, 64, 1040), (33, 300, 144), (48, 1, 2048), (64, 131, 400)])
def test_few_rows(M, N, K, out):
    check(operands(M, N, K, seed=M + N), out)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(65, 1, 16), (128, 128, 128), (129, 257, 144), (300, 1999, 1552), (200, 64, 2048),
                                   (1000, 40, 272), (70, 2560, 2048), (2500, 520, 640)])
def test_many_rows(M, N, K, out):
    check(operands(M, N, K, seed=M + N), out)


@pytest.mark.parametrize("M", [15, 16, 17, 32, 33, 128, 129, 513])
@pytest.mark.parametrize("N,K", [(4100, 2064), (136, 4096), (24, 128)])
def test_every_way_a_product_is_cut(M, N, K):
    """Rows around the choice of kernel, at sizes that take each tile width."""
    check(operands(M, N, K, seed=M), "bf16")


def test_small_and_odd_results():
    for M, N, K in ((1, 3, 16), (2, 1, 16384), (300, 7, 32), (77, 1001, 48), (1025, 1, 16),
                    (1300, 129, 144), (2200000, 1, 16)):
        for out in ("bf16", "f32"):
            check(operands(M, N, K, seed=K), out)


def test_scales_far_apart_and_zero():
    """Block scales over many octaves, zero blocks, and a row and a column of zeros."""
    for M, N, K in ((12, 300, 640), (200, 300, 640)):
        a, sa, b, sb = operands(M, N, K)
        g = torch.Generator(device="cuda").manual_seed(1)
        sa.copy_(torch.exp2(torch.empty_like(sa).uniform_(-40, 20, generator=g)))
        sb.copy_(torch.exp2(torch.empty_like(sb).uniform_(-40, 20, generator=g)))
        sa[3], sb[1, 2], a[5] = 0, 0, 0
        c = check((a, sa, b, sb), "f32")
        assert bool((c[3] == 0).all()) and bool((c[5] == 0).all())


@pytest.mark.parametrize("M", [9, 300])
def test_nan_codes_and_scales_stay_in_their_row_and_column(M):
    N, K = 260, 400
    a, sa, b, sb = operands(M, N, K)
    clean = mxq.gemm_fp8(a, sa, b, sb)["c"]
    a[4, 399], b[130, 7] = 0x7F, 0xFF
    c = mxq.gemm_fp8(a, sa, b, sb)["c"]
    want = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    want[4], want[:, 130] = True, True
    assert torch.equal(torch.isnan(c), want) and torch.equal(c[~want], clean[~want])
    a, sa, b, sb = operands(M, N, K)
    sa[2, 1] = float("nan")
    assert torch.equal(torch.isnan(mxq.gemm_fp8(a, sa, b, sb)["c"]).any(1).nonzero().flatten().cpu(), torch.tensor([2]))


@pytest.mark.parametrize("M,N,K", [(8, 512, 1024), (500, 1000, 1040), (4000, 2560, 2048)])
def test_repeated_streamed_and_captured_calls(M, N, K):
    """The same bits from call to call (many in a row), from two streams at once and from a captured graph."""
    ops = operands(M, N, K)
    c0 = mxq.gemm_fp8(*ops)["c"]
    outs = [mxq.gemm_fp8(*ops) for _ in range(40)]
    assert all(torch.equal(o["c"], c0) and int(o["status"].item()) == 0 for o in outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both = []
    for _ in range(10):
        with torch.cuda.stream(side):
            both.append(mxq.gemm_fp8(*ops, out="f32")["c"])
        both.append(mxq.gemm_fp8(*ops, out="f32")["c"])
    torch.cuda.synchronize()
    assert all(torch.equal(x, both[0]) for x in both)
    c, st = torch.empty_like(c0), torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.mxq_gemm_fp8(*ops, M, N, K, "bf16", c, st)
    new = operands(M, N, K, seed=77)
    for old, t in zip(ops, new):
        old.copy_(t)
    for _ in range(3):
        graph.replay()
    assert torch.equal(c, mxq.gemm_fp8(*new)["c"]) and int(st.item()) == 0


def test_offsets_past_32_bits():
    """Operands and results of more than 2^32 bytes: the first and the last rows and columns."""
    for M, N, K in ((300000, 256, 16384), (600000, 4096, 128)):
        a = torch.randint(0, 0x7E, (M, K), dtype=torch.uint8, device="cuda")
        sa = torch.rand((M, -(-K // 128)), device="cuda")
        _, _, b, sb = operands(1, N, K)
        c = mxq.gemm_fp8(a, sa, b, sb)["c"]
        for r in (slice(M - 300, M), slice(0, 300)):
            ref.close(c[r], *ref.gemm(*(t.cpu().numpy() for t in (a[r], sa[r], b, sb)), "bf16"))
        del a, sa, c
    w = torch.randint(0, 0x7E, (300000, 16384), dtype=torch.uint8, device="cuda")
    sw = torch.rand((-(-300000 // 128), 128), device="cuda")
    a, sa, _, _ = operands(4, 1, 16384)
    c = mxq.gemm_fp8(a, sa, w, sw)["c"]
    cut = 128 * 2340
    assert torch.equal(c[:, cut:], mxq.gemm_fp8(a, sa, w[cut:].contiguous(), sw[2340:].contiguous())["c"])


@pytest.mark.parametrize("M,N,K", [(64, 1536, 2048), (40, 2560, 2064), (120, 2000, 1296), (129, 640, 2192), (64, 512, 8192),
                                   (300, 700, 4112), (1100, 200, 1552), (2000, 2100, 400), (4096, 2560, 272), (2500, 2300, 144)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_shared_steps_and_cut_last_rounds(M, N, K, out):
    """Sizes whose tiles are shared by clusters, and whose last round of tiles is cut; the same bits twice."""
    ops = operands(M, N, K, seed=N)
    c = check(ops, out)
    assert all(torch.equal(mxq.gemm_fp8(*ops, out=out)["c"], c) for _ in range(10))


@pytest.mark.parametrize("M,N,K", [(496, 1001, 16), (388, 700, 48), (77, 98, 5072), (31, 53, 4224), (620, 529, 2064), (416, 1100, 4112),
                                   (9, 33, 1040), (16, 2600, 1168), (700, 310, 272), (260, 1002, 400), (1025, 66, 144)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_short_rows_long_rows_and_even_rows(M, N, K, out):
    """Short and long K with few columns, rows of an even but not 16-byte length, tiles of 128 columns shared by pairs."""
    check(operands(M, N, K, seed=K), out)

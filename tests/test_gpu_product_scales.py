"""Block-FP8 product with block scales near both ends of fp32, on the GPU: the
product of two scales may leave the range of fp32 although the scaled sum of a
block does not.

Bound of an fp32 result, beyond (K + 4) 2^-23 sum |a b| and the last rounding
(layer_ref): below 2^-126 a rounding is off by half of 2^-149 instead, and a
block has at most three of them (the sum times one scale, times the other, and
the addition)."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from mxfp_block_scaled_b200 import layers, mxq

pytestmark = pytest.mark.gpu

# streamed by 8 and 16 warps, 8 to 32 rows at a time; tiles of 64 columns, of 128, of 256 (some cut); tiles shared by clusters
SIZES = [(5, 40, 400), (12, 300, 1296), (33, 300, 144), (1100, 64, 272), (2500, 520, 400), (4096, 2560, 272), (129, 640, 2192),
         (64, 1536, 2048), (64, 512, 4112)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def _codes(g, M, K, lo, hi):
    """E4M3 codes of magnitudes lo .. hi - 1, either sign."""
    mag = torch.randint(lo, hi, (M, K), generator=g, device="cuda")
    return (mag + 128 * torch.randint(0, 2, (M, K), generator=g, device="cuda")).to(torch.uint8)


def _scales(g, shape, lo, hi):
    return torch.exp2(torch.empty(shape, device="cuda").uniform_(lo, hi, generator=g))


def _close(a, sa, b, sb):
    r = mxq.gemm_fp8(a, sa, b, sb, out="f32")
    assert int(r["status"].item()) == 0
    A, SA, B, SB = (t.cpu().numpy() for t in (a, sa, b, sb))
    A = ref.E4M3[A] * ref.spread(SA.astype(np.float64), 1, *A.shape)
    B = ref.E4M3[B] * ref.spread(SB.astype(np.float64), 128, *B.shape)
    want, K = A @ B.T, A.shape[1]
    assert np.abs(want).max() < 2.0 ** 127
    err = (K + 4) * 2.0 ** -23 * (np.abs(A) @ np.abs(B.T))
    ref.close(r["c"], want, err + 2.0 ** -24 * (np.abs(want) + err) + (3 * -(-K // 128) + 1) * 2.0 ** -150)
    return r["c"], want


@pytest.mark.parametrize("M,N,K", SIZES)
def test_scales_whose_product_is_subnormal(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    a, b, kb = _codes(g, M, K, 0x60, 0x7F), _codes(g, N, K, 0x60, 0x7F), -(-K // 128)
    for la, lb in ((-88, -53), (-140, -2), (-20, -122), (-149, 100)):
        sa, sb = _scales(g, (M, kb), la, la + 4), _scales(g, (-(-N // 128), kb), lb, lb + 4)
        sa[1, 0], sb[0, 1] = 0, 0                       # blocks of zeros keep their scale 0
        c, want = _close(a, sa, b, sb)
        assert float(c.abs().max()) > 2.0 ** -126 and np.abs(want).max() > 2.0 ** -126


@pytest.mark.parametrize("M,N,K", SIZES)
def test_scales_whose_product_overflows(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(N)
    a, b, kb = _codes(g, M, K, 1, 4), _codes(g, N, K, 1, 4), -(-K // 128)
    b[3], a[2] = 0, 0x80                                # blocks of zeros under any scale
    for la, lb in ((62, 63), (120, 7), (4, 122)):
        c, _ = _close(a, _scales(g, (M, kb), la, la + 3), b, _scales(g, (-(-N // 128), kb), lb, lb + 3))
        assert bool((c[:, 3] == 0).all()) and bool((c[2] == 0).all())


@pytest.mark.parametrize("M,N,K", SIZES)
def test_blocks_of_either_kind_in_one_row(M, N, K):
    """Scales of all of fp32's octaves from block to block, with codes that keep the sums inside the range."""
    g = torch.Generator(device="cuda").manual_seed(K)
    a, b, kb = _codes(g, M, K, 0, 0x20), _codes(g, N, K, 0, 0x20), -(-K // 128)
    _close(a, _scales(g, (M, kb), -149, 62), b, _scales(g, (-(-N // 128), kb), -149, 62))


@pytest.mark.parametrize("M", [6, 700])
def test_infinite_scales_are_products_as_written(M):
    """Inf times a sum that is not 0 is Inf, times 0 NaN; a NaN scale is NaN; other rows are left alone."""
    K, N = 272, 200
    g = torch.Generator(device="cuda").manual_seed(M)
    a, b = _codes(g, M, K, 0x30, 0x40) & 0x7F, _codes(g, N, K, 0x30, 0x40) & 0x7F
    sa, sb = _scales(g, (M, 3), -3, 3), _scales(g, (2, 3), -3, 3)
    clean = mxq.gemm_fp8(a, sa, b, sb)["c"]
    sa[1, 0], sa[2, 1], b[7, :128] = float("inf"), float("nan"), 0
    want = mxq.gemm_fp8(a, torch.where(torch.isfinite(sa), sa, 1.0), b, sb)["c"]
    c = mxq.gemm_fp8(a, sa, b, sb)["c"]
    assert bool(torch.isinf(c[1, :7]).all()) and bool(torch.isnan(c[1, 7])) and bool(torch.isinf(c[1, 8:]).all())
    assert bool(torch.isnan(c[2]).all())
    keep = [m for m in range(M) if m not in (1, 2)]
    assert torch.equal(c[keep], want[keep]) and torch.equal(c[keep][:, 8:], clean[keep][:, 8:])


@pytest.mark.parametrize("M", [3, 400])
def test_tiny_tokens_against_ordinary_weights(M):
    """What the quantizer itself writes for tokens near the smallest normal numbers."""
    K, N = 640, 300
    g = torch.Generator(device="cuda").manual_seed(M)
    x = (torch.randn((M, K), generator=g, device="cuda") * 1e-36).to(torch.bfloat16)
    w = mxq.quantize_fp8((torch.randn((N, K), generator=g, device="cuda") * 0.02).to(torch.bfloat16), 128)
    t = mxq.quantize_fp8(x)
    c, _ = _close(t["codes"], t["scales"], w["codes"], w["scales"])
    assert torch.equal(layers.fp8_linear(x, w, out="f32")["c"], c)


@pytest.mark.parametrize("M,N,K", SIZES + [(700, 311, 400), (9, 77, 272), (129, 642, 2192)])       # rows of odd and even lengths too
def test_bf16_results_are_the_fp32_ones_rounded(M, N, K):
    """Far scales and ordinary ones, some of the blocks 0: the same sums, rounded once; memory beside the result is left alone."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    a, b, kb, pad = _codes(g, M, K, 0, 0x50), _codes(g, N, K, 0, 0x50), -(-K // 128), 512
    for la, lb in ((-100, -40), (60, 50), (-3, -3)):
        sa, sb = _scales(g, (M, kb), la, la + 4), _scales(g, (-(-N // 128), kb), lb, lb + 4)
        sa[M // 2, kb // 2], sb[0, 0] = 0, 0
        full = torch.full((M * N + 2 * pad,), 3.0, dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        mxq.mxq_gemm_fp8(a, sa, b, sb, M, N, K, "bf16", full[pad:pad + M * N], st)
        c = mxq.gemm_fp8(a, sa, b, sb, out="f32")["c"]
        assert int(st.item()) == 0 and bool(torch.isfinite(c).all())
        assert torch.equal(full[pad:pad + M * N].view(M, N), c.to(torch.bfloat16))
        assert bool((full[:pad] == 3).all()) and bool((full[pad + M * N:] == 3).all())


@pytest.mark.parametrize("M,N,K", [(6, 300, 1296), (700, 310, 2064), (64, 512, 4112)])
def test_far_scales_captured_and_side_by_side(M, N, K):
    """The scales that a replayed graph finds decide, not those of the capture; streams at once.  The largest scales
    overflow some results, so bits are compared."""
    g = torch.Generator(device="cuda").manual_seed(K)
    a, b, kb = _codes(g, M, K, 0, 0x50), _codes(g, N, K, 0, 0x50), -(-K // 128)
    sets = [(_scales(g, (M, kb), la, la + 3), _scales(g, (-(-N // 128), kb), lb, lb + 3)) for la, lb in ((-2, -3), (-95, -50), (58, 62))]
    want = [mxq.gemm_fp8(a, *s[:1], b, s[1], out="f32")["c"] for s in sets]
    sa, sb = (t.clone() for t in sets[0])
    c, st = torch.empty_like(want[0]), torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.mxq_gemm_fp8(a, sa, b, sb, M, N, K, "f32", c, st)
    for i in (1, 0, 2, 1, 0):
        sa.copy_(sets[i][0]), sb.copy_(sets[i][1])
        graph.replay()
        assert torch.equal(c.view(torch.int32), want[i].view(torch.int32))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    outs = [[mxq.gemm_fp8(a, s[0], b, s[1], out="f32", stream=t)["c"] for s, t in zip(sets, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o.view(torch.int32), w.view(torch.int32)) for row in outs for o, w in zip(row, want)) and int(st.item()) == 0

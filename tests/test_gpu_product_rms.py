"""The fp32 result of the block-FP8 product for long K, by the root mean square of its error (product_rms); the
elementwise bound of the other tests does not tell fp32 block sums from bf16 ones there."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import product_rms as pr
from mxfp_block_scaled_b200 import mxq, workloads

# streamed by 8 and 16 warps, 8 to 32 rows at a time; clusters of 4 and 2; tiles of 64, 128 and 256 columns, some cut
SIZES = [(1, 2560, 2048), (8, 1000, 8192), (16, 2048, 1280), (31, 53, 4224), (64, 512, 8192), (64, 1536, 2048), (300, 700, 4112),
         (1100, 200, 1552), (700, 310, 2064), (2500, 1300, 1040)]


def _operands(M, N, K, device):
    w = torch.randn((N, K), generator=torch.Generator().manual_seed(N)) * 0.02
    return workloads.activation_tile(M, seed=K, device="cpu", hidden=K).to(device), w.to(torch.bfloat16).to(device)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
def test_error_of_long_sums(M, N, K):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    x, w = _operands(M, N, K, "cuda")
    a, b = mxq.quantize_fp8(x), mxq.quantize_fp8(w, brows=128)
    ops = a["codes"], a["scales"], b["codes"], b["scales"]
    P, mag = pr.block_sums(*(t.cpu().numpy() for t in ops))
    err = mxq.gemm_fp8(*ops, out="f32")["c"].double().cpu().numpy() - P.sum(0)
    assert pr.rms(err) <= pr.bound(P, mag), (pr.rms(err), pr.bound(P, mag))


@pytest.mark.parametrize("M,N,K", [(8, 100, 8192), (31, 53, 4224), (64, 128, 2048)])
def test_the_bound_tells_block_sums_of_fewer_bits(M, N, K):
    """Planted in the oracle: block sums rounded to fp32 pass, to bf16 they do not (nor does their sum in bf16)."""
    x, w = _operands(M, N, K, "cpu")
    ca, sa = ref.quantize_fp8(x.float().numpy(), 1)
    cb, sb = ref.quantize_fp8(w.float().numpy(), 128)
    P, mag = pr.block_sums(ca, sa, cb, sb)
    limit, t = pr.bound(P, mag), torch.from_numpy(P)
    assert pr.rms(t.float().numpy().sum(0) - P.sum(0)) < limit
    assert pr.rms(t.bfloat16().double().numpy().sum(0) - P.sum(0)) > 3 * limit
    s = torch.zeros_like(t[0])
    for p in t:
        s = (s + p).bfloat16().double()
    assert pr.rms(s.numpy() - P.sum(0)) > 3 * limit

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

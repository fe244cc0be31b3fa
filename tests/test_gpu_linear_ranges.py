"""mxq_linear over its whole range, against binary64: up to 2048 tokens, rows of up to 65536
values (one token a CTA, two slots of a ring), and tokens whose elements lie far apart.

Bounds as in test_gpu_linear.py.  A token's elements are held in f16 relative to its largest,
which stands at 2^14 or above, so each is off by 2^-25 / 2^14 = 2^-39 of the largest at most."""
import pytest
import torch

from mxfp_block_scaled_b200 import mxq
from test_gpu_linear import check, dense, gen, matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,N,K", [(71, 300, 512), (128, 33, 2048), (500, 1000, 96), (1000, 17, 4096), (2047, 50, 256), (2048, 2560, 224),
                                   (33, 100, 8192), (7, 40, 16384), (5, 700, 40000), (1, 20, 65536), (3, 2400, 65536), (2, 16, 65504),
                                   (40, 70, 32800)])
def test_many_tokens_and_long_rows(T, N, K, fmt):
    x = torch.randn((T, K), generator=gen(T + N), device="cuda").bfloat16()
    x *= torch.exp2(torch.randint(-20, 21, (T, 1), generator=gen(K), device="cuda").float()).bfloat16()
    w = matrix(N, K, fmt, N * 7 + K)
    r = mxq.linear(x, w, fmt, out="f32")
    check(r["y"], x, w, "f32")
    assert r["status"].item() == 0 and torch.equal(r["y"], mxq.linear(x, w, fmt, out="f32")["y"])
    check(mxq.linear(x, w, fmt)["y"], x, w, "bf16")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("far", [28, 31, 34, 38, 45])
def test_elements_far_below_a_tokens_largest(far, T, fmt):
    """The largest meets a column of zeros; the others are 2^-far of it."""
    K = 256
    w = matrix(40, K, fmt, 5)
    w["codes"][:, :32 if fmt == "mxfp8" else 16] = 0
    x = torch.randn((T, K), generator=gen(1), device="cuda").bfloat16()
    x[:, 0] = 2.0 ** far
    y = mxq.linear(x, w, fmt, out="f32")["y"].double()
    d = dense(w)
    want, mag = x.double() @ d.t(), x.double().abs() @ d.t().abs()
    bound = mag * (K / 16 + 16) * 2.0 ** -22 + 2.0 ** (far - 39) * d.abs().sum(1)
    assert ((y - want).abs() <= bound).all(), ((y - want).abs() / bound).max().item()

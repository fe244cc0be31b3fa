"""mxq_linear on the GPU against binary64 over the same codes.

Bound of a sum: the tensor core cuts its partial sums (at most 2^-22 of the products'
magnitudes for each of the K / 16 steps of a chain) and the fp32 additions round
(2^-24 each), a rounding to the output's type comes last."""
import pytest
import torch

import cache_ref as ref
from mxfp_block_scaled_b200 import layers, mxq

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(N, K, fmt, seed):
    w = torch.randn((N, K), generator=gen(seed), device="cuda") * 0.05
    w *= torch.exp2(torch.randint(-6, 7, (N, 1), generator=gen(seed + 1), device="cuda").float())
    return layers.quantize_projection(w.bfloat16(), fmt)


def dense(w):
    s2 = w["s2"].expand(w["codes"].shape[0]) if w["fmt"] == "nvfp4" else None
    return ref.values(w["codes"], w["scales"], w["fmt"], s2)


def check(y, x, w, out):
    d = dense(w)
    want, mag = x.double() @ d.t(), x.double().abs() @ d.t().abs()
    bound = want.abs() * HALF[out] * 1.01 + mag * (x.shape[1] / 16 + 16) * 2.0 ** -22 + 1e-30
    worst = ((y.double() - want).abs() / bound).max().item()
    assert worst <= 1, worst


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (1, 2560, 2048), (3, 17, 96), (5, 16, 64), (8, 31, 160), (9, 50, 1120), (17, 33, 416),
                                   (33, 40, 2080), (70, 200, 4096), (1, 50, 12288), (2, 5003, 256), (64, 2048, 128)])
def test_against_binary64(T, N, K, fmt, out):
    x = torch.randn((T, K), generator=gen(T + N), device="cuda").bfloat16()
    x *= torch.exp2(torch.randint(-20, 21, (T, 1), generator=gen(K), device="cuda").float()).bfloat16()
    if T > 2:
        x[1] = 0
    w = matrix(N, K, fmt, N * 7 + K)
    r = mxq.linear(x, w, fmt, out=out)
    check(r["y"], x, w, out)
    assert r["status"].item() == 0
    assert torch.equal(r["y"], mxq.linear(x, w, fmt, out=out)["y"])             # the same bits
    # a token's row does not depend on the others' values
    if T > 2:
        y = mxq.linear(torch.cat((x[:1], x[1:] * 3)), w, fmt, out=out)["y"]
        assert torch.equal(y[:1], r["y"][:1])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("K", [128, 224, 352])
def test_one_hot_tokens_read_the_matrix_exactly(fmt, K):
    w = matrix(45, K, fmt, K)
    y = mxq.linear(torch.eye(K, device="cuda").bfloat16(), w, fmt, out="f32")["y"]
    want = dense(w).t()
    if fmt == "nvfp4":          # code times scale is exact, the product with s2 is rounded once
        want = (want / w["s2"].double()).float() * w["s2"]
    assert torch.equal(y.double(), want.double())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_small_elements_of_a_token_count(fmt):
    """Elements 2^-24 of the largest, which meets a column of zeros."""
    K = 256
    w = matrix(40, K, fmt, 5)
    w["codes"][:, :32 if fmt == "mxfp8" else 16] = 0
    x = torch.randn((4, K), generator=gen(1), device="cuda").bfloat16()
    x[:, 0] = 2.0 ** 24
    check(mxq.linear(x, w, fmt, out="f32")["y"], x, w, "f32")


@pytest.mark.parametrize("T", [3, 40])
def test_a_nonfinite_token_leaves_the_others(T):
    w = matrix(70, 256, "nvfp4", 3)
    x = torch.randn((T, 256), generator=gen(2), device="cuda").bfloat16()
    y = mxq.linear(x, w, "nvfp4")["y"]
    for bad in (float("inf"), float("nan")):
        z = x.clone()
        z[1, 100] = bad
        r = mxq.linear(z, w, "nvfp4")
        assert r["status"].item() == mxq.DEV_NONFINITE_INPUT
        keep = [t for t in range(T) if t != 1]
        assert torch.equal(r["y"][keep], y[keep])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_scales_at_odd_addresses_and_the_end_of_y(fmt):
    w = matrix(21, 256, fmt, 9)
    x = torch.randn((3, 256), generator=gen(2), device="cuda").bfloat16()
    want = mxq.linear(x, w, fmt)["y"]
    shifted = torch.empty(w["scales"].numel() + 1, dtype=torch.uint8, device="cuda")
    shifted[1:] = w["scales"].flatten()
    y = torch.full((3 * 21 + 64,), 7.0, device="cuda", dtype=torch.bfloat16)
    st, ws = torch.zeros(1, dtype=torch.int32, device="cuda"), mxq.linear_workspace(3, 256)
    mxq.mxq_linear(x, 3, 256, fmt, w["codes"], shifted[1:], w.get("s2"), 21, "bf16", y, st, ws)
    assert torch.equal(y[:63].view(3, 21), want) and (y[63:] == 7).all()


def test_hundreds_of_millions_of_rows():
    """16-row tasks times CTAs past 32 bits, and codes past the fourth gibibyte."""
    N, K = 480_000_007, 32
    codes = torch.empty((N, 16), dtype=torch.uint8, device="cuda").random_(generator=gen(1))
    scales = torch.empty((N, 1), dtype=torch.uint8, device="cuda").random_(120, 131, generator=gen(2))
    x = torch.randn((1, K), generator=gen(3), device="cuda").bfloat16()
    y = mxq.linear(x, {"codes": codes, "scales": scales}, "mxfp4")["y"][0]
    rows = torch.cat((torch.arange(64), torch.arange(N - 64, N), torch.randint(0, N, (20000,), generator=torch.Generator().manual_seed(4)))).cuda()
    check(y[rows][None], x, {"codes": codes[rows], "scales": scales[rows], "fmt": "mxfp4"}, "bf16")


def test_empty_sizes():
    w = {"codes": torch.empty((9, 0), dtype=torch.uint8, device="cuda"), "scales": torch.empty((9, 0), dtype=torch.uint8, device="cuda")}
    x = torch.empty((2, 0), dtype=torch.bfloat16, device="cuda")
    y = torch.ones((2, 9), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mxq.mxq_linear(x, 2, 0, "mxfp8", w["codes"], w["scales"], None, 9, "f32", y, st, None)
    assert (y == 0).all()
    w = matrix(16, 64, "mxfp8", 1)
    assert mxq.linear(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w, "mxfp8")["y"].shape == (0, 16)


def test_more_tokens_than_a_call_takes_are_refused():
    w = matrix(16, 64, "mxfp8", 1)
    with pytest.raises(mxq.MxqError, match="unsupported"):
        mxq.linear(torch.zeros((2049, 64), dtype=torch.bfloat16, device="cuda"), w, "mxfp8")


@pytest.mark.parametrize("T", [2, 40])
def test_captured_replayed_and_side_by_side(T):
    """Two calls in one graph, on two streams, each with its own workspace; replays see new
    tokens."""
    ws = [matrix(300, 512, f, 2) for f in ("nvfp4", "mxfp8")]
    x = torch.randn((T, 512), generator=gen(4), device="cuda").bfloat16()
    work = [mxq.linear_workspace(T, 512) for _ in ws]
    y = [torch.empty((T, 300), device="cuda") for _ in ws]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def go(i, stream=None):
        w = ws[i]
        mxq.mxq_linear(x, T, 512, w["fmt"], w["codes"], w["scales"], w.get("s2"), 300, "f32", y[i], st, work[i], stream)
    go(0), go(1)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        go(0)
        go(1, side)
        torch.cuda.current_stream().wait_stream(side)
    for seed in (5, 6):
        x.copy_(torch.randn((T, 512), generator=gen(seed), device="cuda"))
        graph.replay()
        for i, w in enumerate(ws):
            assert torch.equal(y[i], mxq.linear(x, w, w["fmt"], out="f32")["y"])

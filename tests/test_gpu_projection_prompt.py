"""Projections of prompts: more tokens than a call of mxq_linear takes go through it in pieces,
and from the projections into the cache and its attention."""
import pytest
import torch

from mxfp_block_scaled_b200 import layers, mxq
from test_gpu_cache import dev32
from test_gpu_linear import check, gen, matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("T", [2048, 2049, 4096, 5001])
def test_prompts_of_any_length(T, fmt, out):
    w = matrix(96, 256, fmt, 3)
    x = torch.randn((T, 256), generator=gen(T), device="cuda").bfloat16()
    r = layers.projection_forward(w, x, out=out)
    check(r["y"], x, w, out)
    assert r["status"].item() == 0
    ws = mxq.linear_workspace(mxq.LINEAR_MAX_TOKENS, 256)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    again = layers.projection_forward(w, x, out=out, workspace=ws, stream=stream)
    stream.synchronize()
    assert torch.equal(again["y"], r["y"])
    x[T - 1, 3] = float("inf")          # of the last piece
    z = layers.projection_forward(w, x, out=out)
    assert z["status"].item() == mxq.DEV_NONFINITE_INPUT and torch.equal(z["y"][:-1], r["y"][:-1])


def test_a_given_result_of_another_shape_is_refused():
    w = matrix(96, 256, "mxfp8", 3)
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    for y in (torch.zeros((4, 96), device="cuda"), torch.zeros((5, 96), dtype=torch.bfloat16, device="cuda"),
              torch.zeros((96, 4), dtype=torch.bfloat16, device="cuda").t()):
        with pytest.raises(ValueError):
            mxq.linear(x, w, "mxfp8", y=y)


def test_a_chunk_of_4096_tokens_through_the_layer():
    """Projection, cache, attention and output projection of a prompt in one piece, as in two."""
    H, heads, kv, dim, T = 128, 4, 2, 64, 4096
    w_qkv = layers.quantize_projection(torch.randn(((heads + 2 * kv) * dim, H), generator=gen(1), device="cuda").bfloat16() * 0.08, "mxfp8")
    x = torch.randn((T, H), generator=gen(2), device="cuda").bfloat16()
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    outs = []
    for cuts in ((0, T), (0, 2000, T)):
        cache = mxq.Cache.empty(64, kv, 64, dim)
        o = []
        for t0, t1 in zip(cuts, cuts[1:]):
            qkv = layers.projection_forward(w_qkv, x[t0:t1])["y"].view(t1 - t0, heads + 2 * kv, dim)
            r = layers.attention_forward(cache, qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:],
                                         dev32([0, t1 - t0]), dev32([t1]), table, t1 - t0)
            assert r["status"].item() == 0
            o.append(r["o"])
        outs.append(torch.cat(o).float())
    # the same keys and values; each output within 2^-8 of itself and 2^-10 of the values, which are below 8
    assert ((outs[0] - outs[1]).abs() <= 2.0 ** -7 * outs[0].abs() + 2.0 ** -6).all()

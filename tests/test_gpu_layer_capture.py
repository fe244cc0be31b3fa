"""The layer operators in captured graphs whose nodes before and after them are not their own: fills, copies, torch
kernels, and branches that fork from and join the capturing stream."""
import pytest
import torch

from mxfp_block_scaled_b200 import layers, mxq, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def test_fills_copies_and_branches_around_the_operators():
    E, H, I, T, k = 8, 512, 256, 20, 3
    L = layers.quantize_routed_layer(*workloads.tiny_moe_layer(seed=5, device="cuda", experts=E, hidden=H, inter=I), fmt="mxfp4")
    w_q = mxq.quantize_fp8(torch.randn((700, H), device="cuda").to(torch.bfloat16), 128)
    gate = torch.randn((H, E), device="cuda")
    x_in, x = (workloads.activation_tile(T, seed=1, device="cuda", hidden=H) for _ in range(2))
    out = {}

    def step(side):
        x.copy_(x_in)                                           # a copy before
        main = torch.cuda.current_stream()
        side.wait_stream(main)                                  # a branch: the product beside the layer
        with torch.cuda.stream(side):
            c = layers.fp8_linear(x, w_q)["c"]
            many = layers.fp8_linear(x.repeat(40, 1), w_q, out="f32")["c"]
        top = torch.softmax(x.float() @ gate, -1).topk(k, -1)
        y = layers.routed_forward(L, x, top.indices.int().contiguous(), top.values.contiguous())["y"]
        main.wait_stream(side)
        out["z"] = (c.float().sum(1) + y.float().sum(1), c, y, many)
        zero = layers.fp8_linear(x[:, :0].contiguous(), {"codes": w_q["codes"][:, :0].contiguous(),
                                                         "scales": w_q["scales"][:, :0].contiguous()})["c"]   # a fill
        again = layers.fp8_linear(x, w_q)["c"]
        out["end"] = (zero, again)

    side = torch.cuda.Stream()
    step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(side)
    got = out["z"] + out["end"]
    for seed in range(5):
        x_in.copy_(workloads.activation_tile(T, seed=seed, device="cuda", hidden=H))
        for _ in range(3):
            graph.replay()
        held = [t.clone() for t in got]
        step(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, out["z"] + out["end"]))

"""The layer operators as a model uses them, on the GPU: converted layers run
from the codes they are stored in, a routed block with a shared expert, calls
side by side and captured."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from mxfp_block_scaled_b200 import layers, mxq, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def router(x, gate, k):
    top = torch.softmax(x.float() @ gate, -1).topk(k, -1)
    return top.indices.int().contiguous(), (top.values / top.values.sum(-1, keepdim=True)).contiguous()


def np_(t):
    return t.cpu().numpy()


def linear_ref(x, w_q, out):
    """(codes and scales are the definition's, bit for bit) -> (c, bound)."""
    a, sa = ref.quantize_fp8(np_(x.float()), 1)
    return ref.gemm(a, sa, np_(w_q["codes"]), np_(w_q["scales"]), out)


@pytest.mark.parametrize("T", [1, 7, 64])
def test_a_mixed_model_from_conversion_to_tokens(T):
    """Layers in the four formats a mixed model holds, each with a shared expert
    in block FP8: convert, route, run, against binary64 on the same codes."""
    E, H, I, k = 12, 384, 256, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    gate = torch.randn((H, E), generator=g, device="cuda") / H ** 0.5
    stacks = [workloads.tiny_moe_layer(seed=i, device="cuda", experts=E, hidden=H, inter=I) for i in range(4)]
    model = layers.quantize_mixed(stacks[:3], ["nvfp4", "mxfp4", "mxfp8"]) + [layers.block_fp8_layer(*stacks[3])]
    ws = mxq.moe_workspace(T, k, H, I)
    for i, layer in enumerate(model):
        x = workloads.activation_tile(T, seed=i, device="cuda", hidden=H)
        s_gu, s_dn = workloads.tiny_moe_layer(seed=40 + i, device="cuda", experts=1, hidden=H, inter=I)
        w_gu, w_dn = mxq.quantize_fp8(s_gu[0], 128), mxq.quantize_fp8(s_dn[0], 128)
        ids, w = router(x, gate, k)
        routed = layers.routed_forward(layer, x, ids, w, workspace=ws)
        want, bound = ref.moe(x, ids, w, layer["gate_up"], layer["down"], layer["gate_up"]["fmt"])
        ref.close(routed["y"], want, bound)
        # the shared expert: products on quantized tokens
        a = layers.fp8_linear(x, w_gu, out="f32")
        want, bound = linear_ref(x, w_gu, "f32")
        ref.close(a["c"], want, bound)
        h = (torch.nn.functional.silu(a["c"][:, :I]) * a["c"][:, I:]).to(torch.bfloat16)
        z = layers.fp8_linear(h, w_dn)
        want, bound = linear_ref(h, w_dn, "bf16")
        ref.close(z["c"], want, bound)
        for r in (routed, a, z):
            assert int(r["status"].item()) == 0
        # the same expert without quantizing the tokens: one expert of a routed layer
        one = layers.block_fp8_layer(s_gu, s_dn)
        ids1, w1 = torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.ones((T, 1), device="cuda")
        y = layers.routed_forward(one, x, ids1, w1)["y"].double()
        # tokens and h rounded to E4M3 (2^-4 of a value, or of the block's scale below its normals):
        # a few per cent of the result's norm, far from the two being different weights
        assert float((y - z["c"].double()).norm() / y.norm()) < 2.0 ** -4 * 2.5


def test_nonfinite_tokens_are_reported_by_both_steps():
    H, N = 256, 200
    w = mxq.quantize_fp8(torch.randn((N, H), device="cuda").to(torch.bfloat16), 128)
    x = workloads.activation_tile(6, seed=0, device="cuda", hidden=H)
    clean = layers.fp8_linear(x, w)["c"]
    x[2, 200] = float("inf")
    r = layers.fp8_linear(x, w)
    assert int(r["status"].item()) == mxq.DEV_NONFINITE_INPUT
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(r["c"][keep], clean[keep])


def _layer(E=16, H=512, I=256, fmt="mxfp4"):
    return layers.quantize_routed_layer(*workloads.tiny_moe_layer(seed=5, device="cuda", experts=E, hidden=H, inter=I),
                                        fmt=fmt)


def test_two_calls_at_once():
    """Different tokens on two streams, many times over, each with a workspace of its own."""
    L, E, H, k = _layer(), 16, 512, 4
    gate = torch.randn((H, E), device="cuda")
    cases = []
    for T in (3, 40):
        x = workloads.activation_tile(T, seed=T, device="cuda", hidden=H)
        ids, w = router(x, gate, k)
        cases.append((x, ids, w, mxq.moe_workspace(T, k, H, 256), layers.routed_forward(L, x, ids, w)["y"]))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (x, ids, w, ws, _) in enumerate(cases):
            got[i].append(layers.routed_forward(L, x, ids, w, workspace=ws, stream=streams[i])["y"])
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        assert all(torch.equal(y, c[4]) for y in got[i])


def test_a_stream_that_is_not_the_current_one():
    """Results and workspaces belong to the given stream: memory freed on return is not handed to the current one early."""
    L, H = _layer(), 512
    x = workloads.activation_tile(48, seed=1, device="cuda", hidden=H)
    ids, w = router(x, torch.randn((H, 16), device="cuda"), 4)
    y0 = layers.routed_forward(L, x, ids, w)["y"]
    wq = mxq.quantize_fp8(torch.randn((300, H), device="cuda").to(torch.bfloat16), 128)
    c0 = layers.fp8_linear(x, wq)["c"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        y = layers.routed_forward(L, x, ids, w, stream=side)
        junk = torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
        c = layers.fp8_linear(x, wq, stream=side)
        junk = torch.full((1 << 16,), -1, dtype=torch.int32, device="cuda")
        side.synchronize()
        assert torch.equal(y["y"], y0) and torch.equal(c["c"], c0)
        assert int(y["status"].item()) == 0 and int(c["status"].item()) == 0
    del junk


def test_two_captured_graphs_that_share_a_workspace():
    """Replayed one behind the other on one stream, the second call's use of the workspace waits for the first's."""
    L, E, H, I, k = _layer(), 16, 512, 256, 4
    gate = torch.randn((H, E), device="cuda")
    ws = mxq.moe_workspace(64, k, H, I)
    graphs = []
    for T in (64, 2):
        x = workloads.activation_tile(T, seed=T, device="cuda", hidden=H)
        ids, w = router(x, gate, k)
        want = layers.routed_forward(L, x, ids, w)["y"]
        gu, dn = L["gate_up"], L["down"]
        y, st = torch.empty_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                mxq.mxq_moe_forward(x, T, H, ids, w, k, "mxfp4", E, I, gu["codes"], gu["scales"], None, dn["codes"],
                                    dn["scales"], None, y, st, ws)
        graphs.append((graph, y, want, (x, ids, w, st)))
    for _ in range(25):
        for g in graphs:
            g[1].fill_(7)
            g[0].replay()
        for g in graphs:
            g[0].replay()
        assert all(torch.equal(g[1], g[2]) for g in graphs)


def test_empty_tiles():
    L, H = _layer(), 512
    e = layers.routed_forward(L, torch.empty((0, H), dtype=torch.bfloat16, device="cuda"),
                              torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda"))
    assert tuple(e["y"].shape) == (0, H)
    x = workloads.activation_tile(3, seed=1, device="cuda", hidden=H)
    e = layers.routed_forward(L, x, torch.empty((3, 0), dtype=torch.int32, device="cuda"), torch.empty((3, 0), device="cuda"))
    assert bool((e["y"] == 0).all())
    wq = mxq.quantize_fp8(torch.randn((130, H), device="cuda").to(torch.bfloat16), 128)
    assert tuple(layers.fp8_linear(x[:0], wq)["c"].shape) == (0, 130)
    none = mxq.quantize_fp8(torch.empty((130, 0), dtype=torch.bfloat16, device="cuda"), 128)
    c = layers.fp8_linear(torch.empty((3, 0), dtype=torch.bfloat16, device="cuda"), none)["c"]
    assert tuple(c.shape) == (3, 130) and bool((c == 0).all())


def test_layer_operators_write_only_what_they_own():
    """Rows behind the last token, and memory on both sides of every output, stay as they were."""
    T, H, N, pad = 5, 384, 200, 512
    x = workloads.activation_tile(T, seed=3, device="cuda", hidden=H)
    wq = mxq.quantize_fp8(torch.randn((N, H), device="cuda").to(torch.bfloat16), 128)
    codes = torch.full((T * H + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((T * 3 + 2 * pad,), 9.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mxq.mxq_quantize_fp8(x, T, H, 1, 128, codes[pad:pad + T * H], scales[pad:pad + 3 * T], st)
    want = mxq.quantize_fp8(x)
    assert torch.equal(codes[pad:-pad].view(T, H), want["codes"]) and torch.equal(scales[pad:-pad].view(T, 3), want["scales"])
    assert all(bool((t[:pad] == t[0]).all() and (t[-pad:] == t[0]).all()) for t in (codes, scales))
    for rows in (T, 300):
        q = mxq.quantize_fp8(workloads.activation_tile(rows, seed=3, device="cuda", hidden=H))
        for out, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
            c = torch.full((rows * N + 2 * pad,), 3.0, dtype=dt, device="cuda")
            mxq.mxq_gemm_fp8(q["codes"], q["scales"], wq["codes"], wq["scales"], rows, N, H, out, c[pad:pad + rows * N], st)
            assert torch.equal(c[pad:-pad].view(rows, N), mxq.gemm_fp8(q["codes"], q["scales"], wq["codes"], wq["scales"], out)["c"])
            assert bool((c[:pad] == 3).all() and (c[-pad:] == 3).all())
    assert int(st.item()) == 0 and np.isfinite(float(c.float().sum()))

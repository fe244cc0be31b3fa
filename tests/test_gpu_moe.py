"""The mixture-of-experts layer for a few tokens on the GPU against its
definition in binary64, elementwise inside a bound derived from the kernels'
roundings (layer_ref)."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from mxfp_block_scaled_b200 import mxq, workloads

pytestmark = pytest.mark.gpu

FMTS = ["nvfp4", "mxfp4", "mxfp8", "fp8_block"]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def stacks(fmt, E, H, I, seed=0):
    gu, dn = workloads.tiny_moe_layer(seed=seed, device="cuda", experts=E, hidden=H, inter=I)
    q = {"nvfp4": lambda x: mxq.quantize_nvfp4(x), "fp8_block": lambda x: mxq.quantize_fp8(x, 128)}.get(
        fmt, lambda x: mxq.quantize_mx(x, fmt))
    return q(gu), q(dn)


def routing(T, k, E, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    top = torch.randn((T, E), generator=g, device="cuda").topk(k, 1)
    return top.indices.int().contiguous(), torch.softmax(top.values, 1).contiguous()


def check(x, ids, w, gu, dn, fmt):
    out = mxq.moe_forward(x, ids, w, gu, dn, fmt)
    want, bound = ref.moe(x, ids, w, gu, dn, fmt)
    ref.close(out["y"], want, bound)
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 128, 128), (1, 2, 8, 256, 128), (3, 4, 8, 384, 256), (5, 4, 8, 256, 128),
                                       (8, 4, 16, 512, 384), (9, 5, 7, 640, 128), (33, 2, 4, 256, 256),
                                       (64, 10, 40, 256, 128), (1, 10, 16, 2048, 768)])
def test_layer(fmt, T, k, E, H, I):
    gu, dn = stacks(fmt, E, H, I, seed=T + H)
    x = workloads.activation_tile(T, seed=T, device="cuda", hidden=H)
    out = check(x, *routing(T, k, E, seed=T), gu, dn, fmt)
    assert int(out["status"].item()) == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8_block"])
@pytest.mark.parametrize("H,I", [(4096, 128), (128, 4096), (8192, 128), (128, 8192)])
def test_wide_layers(fmt, H, I):
    """Widths whose activation rows leave room for the shorter ring of weights."""
    gu, dn = stacks(fmt, 3, H, I, seed=H)
    x = workloads.activation_tile(9, seed=H, device="cuda", hidden=H)
    check(x, *routing(9, 2, 3, seed=1), gu, dn, fmt)


@pytest.mark.parametrize("T", [3, 40])          # both ways the experts are listed
def test_rows_without_experts_and_repeated_experts(T):
    E, H, I, k = 6, 256, 128, 4
    gu, dn = stacks("mxfp4", E, H, I)
    x = workloads.activation_tile(T, seed=2, device="cuda", hidden=H)
    ids, w = routing(T, k, E)
    ids[0] = -1                                  # a row without a token
    ids[1, 1:] = -5                              # a single expert
    ids[2] = 3                                   # the same expert four times
    x[0] = float("nan")                          # never read: no expert asks for it
    out = check(torch.nan_to_num(x), ids, w, gu, dn, "mxfp4")
    nan = mxq.moe_forward(x, ids, w, gu, dn, "mxfp4")
    assert torch.equal(nan["y"], out["y"]) and int(nan["status"].item()) == 0
    assert bool((out["y"][0] == 0).all())
    ids[:] = -1
    assert bool((mxq.moe_forward(x, ids, w, gu, dn, "mxfp4")["y"] == 0).all())


@pytest.mark.parametrize("T", [3, 40])
def test_invalid_expert_is_reported_and_left_out(T):
    E, H, I, k = 6, 256, 128, 2
    gu, dn = stacks("nvfp4", E, H, I)
    x = workloads.activation_tile(T, seed=2, device="cuda", hidden=H)
    ids, w = routing(T, k, E)
    ids[1, 0] = E
    ids[2, 1] = 2 ** 31 - 1
    out = check(x, ids, w, gu, dn, "nvfp4")
    assert int(out["status"].item()) == mxq.DEV_INVALID_EXPERT


def test_nonfinite_token_leaves_the_others_alone():
    E, H, I, k, T = 4, 256, 128, 2, 12
    gu, dn = stacks("mxfp8", E, H, I)
    x = workloads.activation_tile(T, seed=2, device="cuda", hidden=H)
    ids, w = routing(T, k, E)
    clean = mxq.moe_forward(x, ids, w, gu, dn, "mxfp8")["y"]
    x[5, 17] = float("inf")
    x[7, 0] = float("nan")
    out = mxq.moe_forward(x, ids, w, gu, dn, "mxfp8")
    assert int(out["status"].item()) == mxq.DEV_NONFINITE_INPUT
    keep = [t for t in range(T) if t not in (5, 7)]
    assert torch.equal(out["y"][keep], clean[keep])
    assert not bool(torch.isfinite(out["y"][7].float()).any())


@pytest.mark.parametrize("fmt", FMTS)
def test_extreme_scales_and_tokens(fmt):
    """Block scales far apart inside a row, tokens of very large, very small and
    zero size, and rows whose elements span many octaves."""
    E, H, I, T, k = 3, 256, 256, 7, 2
    gu, dn = stacks(fmt, E, H, I)
    g = torch.Generator(device="cuda").manual_seed(3)
    for q in (gu, dn):
        if fmt == "nvfp4":
            q["scales"].random_(0, 0x7F, generator=g)
            q["s2"].uniform_(1e-6, 1e-2, generator=g)
        elif fmt == "fp8_block":
            q["scales"].copy_(torch.exp2(torch.empty_like(q["scales"]).uniform_(-30, 0, generator=g)))
        else:
            q["scales"].random_(60, 140, generator=g)
            q["scales"].view(-1)[:7] = torch.tensor([0, 1, 2, 100, 0, 127, 128], dtype=torch.uint8)
    x = torch.randn((T, H), generator=g, device="cuda")
    x *= torch.tensor([1e-30, 1e-12, 1.0, 1e6, 0.0, 1.0, 1e-38], device="cuda")[:, None]
    x[5] *= torch.exp2(torch.randint(-30, 10, (H,), generator=g, device="cuda").float())
    check(x.to(torch.bfloat16), *routing(T, k, E), gu, dn, fmt)


def test_nan_codes_of_an_expert_give_nan_there_only():
    E, H, I, T = 4, 256, 128, 4
    gu, dn = stacks("fp8_block", E, H, I)
    x = workloads.activation_tile(T, seed=2, device="cuda", hidden=H)
    ids = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
    w = torch.ones((T, 1), device="cuda")
    clean = mxq.moe_forward(x, ids, w, gu, dn, "fp8_block")["y"]
    dn["codes"][2, 9, 30] = 0x7F
    y = mxq.moe_forward(x, ids, w, gu, dn, "fp8_block")["y"]
    assert bool(torch.isnan(y[2, 9])) and int(torch.isnan(y.float()).sum()) == 1
    y[2, 9] = clean[2, 9]
    assert torch.equal(y, clean)


def test_many_assignments():
    """The largest number of assignments, far more than eight to an expert, and more experts than that."""
    for T, k, E in ((2048, 1, 3), (256, 8, 2000), (204, 10, 10)):
        gu, dn = stacks("nvfp4", E, 128, 128)
        x = workloads.activation_tile(T, seed=2, device="cuda", hidden=128)
        ids, w = routing(T, k, E)
        full = mxq.moe_forward(x, ids, w, gu, dn, "nvfp4")["y"]
        rows = torch.randperm(T, generator=torch.Generator().manual_seed(1))[:24]
        want, bound = ref.moe(x[rows], ids[rows], w[rows], gu, dn, "nvfp4")
        ref.close(full[rows], want, bound)
        # a token's row does not depend on its company
        few = mxq.moe_forward(x[:2].contiguous(), ids[:2].contiguous(), w[:2].contiguous(), gu, dn, "nvfp4")["y"]
        a, b = few.double(), full[:2].double()
        assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -7 * b.abs().max() * 2.0 ** -8).all())


def test_full_size_stack_offsets():
    """The last experts of a stack whose codes pass 2^31 bytes."""
    E, H, I = 1024, 2048, 768
    gu, dn = {}, {}
    for q, R, C in ((gu, 2 * I, H), (dn, H, I)):
        q["codes"] = torch.zeros((E, R, C), dtype=torch.uint8, device="cuda")
        q["scales"] = torch.zeros((E, R, C // 32), dtype=torch.uint8, device="cuda")
        t = mxq.quantize_mx((torch.randn((2, R, C), device="cuda") * 0.02).to(torch.bfloat16), "mxfp8")
        q["codes"][-2:], q["scales"][-2:] = t["codes"], t["scales"]
    x = workloads.activation_tile(3, seed=2, device="cuda", hidden=H)
    ids = torch.tensor([[E - 1, 0], [E - 2, E - 1], [7, E - 2]], dtype=torch.int32, device="cuda")
    w = torch.rand((3, 2), device="cuda")
    small = [{k: torch.cat((q[k][:1], q[k][-2:])) for k in ("codes", "scales")} for q in (gu, dn)]
    ids2 = torch.tensor([[2, 0], [1, 2], [0, 1]], dtype=torch.int32, device="cuda")
    assert torch.equal(check(x, ids2, w, *small, "mxfp8")["y"], mxq.moe_forward(x, ids, w, gu, dn, "mxfp8")["y"])


def test_repeated_streamed_and_captured_calls():
    """The same bits from call to call, on another stream, and from a captured graph whose inputs change."""
    E, H, I, T, k = 16, 512, 256, 12, 4
    gu, dn = stacks("nvfp4", E, H, I)
    x = workloads.activation_tile(T, seed=2, device="cuda", hidden=H)
    ids, w = routing(T, k, E)
    y0 = mxq.moe_forward(x, ids, w, gu, dn, "nvfp4")["y"]
    for _ in range(5):
        assert torch.equal(mxq.moe_forward(x, ids, w, gu, dn, "nvfp4")["y"], y0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1 = mxq.moe_forward(x, ids, w, gu, dn, "nvfp4")["y"]
    y2 = mxq.moe_forward(x, ids, w, gu, dn, "nvfp4")["y"]
    side.synchronize()
    assert torch.equal(y1, y0) and torch.equal(y2, y0)
    y, st = torch.empty_like(y0), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = mxq.moe_workspace(T, k, H, I)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.mxq_moe_forward(x, T, H, ids, w, k, "nvfp4", E, I, gu["codes"], gu["scales"], gu["s2"], dn["codes"],
                            dn["scales"], dn["s2"], y, st, ws)
    ws.fill_(0xFF)
    graph.replay()
    assert torch.equal(y, y0)
    x2 = workloads.activation_tile(T, seed=9, device="cuda", hidden=H)
    ids2, w2 = routing(T, k, E, seed=9)
    want = mxq.moe_forward(x2, ids2, w2, gu, dn, "nvfp4")["y"]
    x.copy_(x2)
    ids.copy_(ids2)
    w.copy_(w2)
    for _ in range(3):
        graph.replay()
    assert torch.equal(y, want)


def test_outputs_stay_inside_their_buffers():
    E, H, I, T, k, pad = 6, 384, 128, 5, 3, 256
    gu, dn = stacks("nvfp4", E, H, I)
    x = workloads.activation_tile(T, seed=2, device="cuda", hidden=H)
    ids, w = routing(T, k, E)
    nb = mxq.moe_workspace(T, k, H, I).numel()
    ws = torch.full((nb + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    yf = torch.full((T * H + 2 * pad,), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mxq.mxq_moe_forward(x, T, H, ids, w, k, "nvfp4", E, I, gu["codes"], gu["scales"], gu["s2"], dn["codes"],
                        dn["scales"], dn["s2"], yf[pad:pad + T * H], st, ws[256:256 + nb])
    assert torch.equal(yf[pad:-pad].view(T, H), mxq.moe_forward(x, ids, w, gu, dn, "nvfp4")["y"])
    assert bool((yf[:pad] == 3).all()) and bool((yf[-pad:] == 3).all())
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[-256:] == 0xA5).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 8, 256, 128), (1, 8, 8, 1024, 512), (4, 2, 8, 2560, 128), (8, 1, 1, 2048, 1280),
                                       (16, 2, 2, 256, 256), (3, 10, 4, 128, 640), (32, 1, 3, 4096, 128), (6, 5, 4, 4864, 384)])
def test_small_layers(fmt, T, k, E, H, I):
    """Few tasks: warps that share a row, tiles summed inside a CTA, several tiles to a CTA; rows without an expert."""
    gu, dn = stacks(fmt, E, H, I, seed=T)
    x = workloads.activation_tile(T, seed=T, device="cuda", hidden=H)
    g = torch.Generator(device="cuda").manual_seed(H)
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, generator=g, device="cuda")
    ids[T // 2, k // 2:] = -1
    if T > 2:
        ids[0] = E - 1
    out = check(x, ids, torch.rand((T, k), generator=g, device="cuda"), gu, dn, fmt)
    assert int(out["status"].item()) == 0
    ids[0, 0] = E
    assert int(check(x, ids, torch.ones((T, k), device="cuda"), gu, dn, fmt)["status"].item()) == mxq.DEV_INVALID_EXPERT
    ids[:] = -7
    assert bool((mxq.moe_forward(x, ids, torch.ones((T, k), device="cuda"), gu, dn, fmt)["y"] == 0).all())


@pytest.mark.parametrize("T,k,E", [(33, 1, 4), (16, 4, 3), (13, 5, 70), (64, 2, 5), (43, 3, 11), (128, 2, 7), (32, 8, 4000), (51, 5, 2), (257, 1, 9)])
def test_every_way_the_experts_are_listed(T, k, E):
    """33 to 257 assignments with few, many and repeated experts, empty and invalid places."""
    gu, dn = stacks("mxfp4", E, 128, 128, seed=E)
    x = workloads.activation_tile(T, seed=T, device="cuda", hidden=128)
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, generator=g, device="cuda")
    ids[T // 3: T // 2] = E - 1
    w = torch.rand((T, k), generator=g, device="cuda")
    out = check(x, ids, w, gu, dn, "mxfp4")
    assert int(out["status"].item()) == 0
    assert torch.equal(out["y"], mxq.moe_forward(x, ids, w, gu, dn, "mxfp4")["y"])
    ids[T - 1, k - 1] = E + 5
    assert int(check(x, ids, w, gu, dn, "mxfp4")["status"].item()) == mxq.DEV_INVALID_EXPERT


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I", [(60, 1, 5, 256, 128), (33, 3, 4, 640, 384), (64, 4, 6, 2048, 128), (90, 1, 1, 384, 256),
                                       (30, 1, 2, 128, 896), (47, 5, 13, 128, 128), (52, 2, 3, 1920, 256)])
def test_many_assignments_to_an_expert(fmt, T, k, E, H, I):
    """Many groups to an expert, the last of any size; some experts without any."""
    gu, dn = stacks(fmt, E, H, I, seed=T)
    x = workloads.activation_tile(T, seed=T, device="cuda", hidden=H)
    g = torch.Generator(device="cuda").manual_seed(H)
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, generator=g, device="cuda")
    ids[ids == E // 2] = 0
    ids[:9] = E - 1
    w = torch.rand((T, k), generator=g, device="cuda")
    out = check(x, ids, w, gu, dn, fmt)
    assert int(out["status"].item()) == 0
    for _ in range(5):
        assert torch.equal(out["y"], mxq.moe_forward(x, ids, w, gu, dn, fmt)["y"])

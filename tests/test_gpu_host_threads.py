"""Calls from several host threads at once, each on a stream and a workspace of its own."""
import threading

import pytest
import torch

from mxfp_block_scaled_b200 import layers, mxq, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def _together(jobs, rounds):
    """Runs every job (a function without arguments) `rounds` times in a thread of its own, all at once."""
    failed, start = [], threading.Barrier(len(jobs))

    def go(job):
        try:
            start.wait(timeout=60)
            for _ in range(rounds):
                job()
        except Exception as e:      # noqa: BLE001 -- reported by the test
            failed.append(repr(e))
    threads = [threading.Thread(target=go, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    torch.cuda.synchronize()
    assert not failed, failed[:3]


def test_layers_of_different_sizes_at_once():
    """Token counts that share a kernel and need different amounts of shared memory."""
    E, H, I, k = 24, 2048, 768, 10
    L = layers.quantize_routed_layer(*workloads.tiny_moe_layer(seed=2, device="cuda", experts=E, hidden=H, inter=I))
    gu, dn = L["gate_up"], L["down"]
    jobs, results = [], []
    for T in (2, 16, 4, 24):
        g = torch.Generator(device="cuda").manual_seed(T)
        x = workloads.activation_tile(T, seed=T, device="cuda", hidden=H)
        top = torch.randn((T, E), generator=g, device="cuda").topk(k, 1)
        ids, w = top.indices.int().contiguous(), torch.softmax(top.values, 1).contiguous()
        want = layers.routed_forward(L, x, ids, w)["y"]
        y, st, ws = torch.empty_like(want), torch.zeros(1, dtype=torch.int32, device="cuda"), mxq.moe_workspace(T, k, H, I)

        def job(x=x, T=T, ids=ids, w=w, y=y, st=st, ws=ws, stream=torch.cuda.Stream()):
            mxq.mxq_moe_forward(x, T, H, ids, w, k, "nvfp4", E, I, gu["codes"], gu["scales"], gu["s2"], dn["codes"],
                                dn["scales"], dn["s2"], y, st, ws, stream=stream)
        jobs.append(job)
        results.append((y, want, st))
    torch.cuda.synchronize()
    _together(jobs, 1500)
    for y, want, st in results:
        assert torch.equal(y, want) and int(st.item()) == 0


@pytest.mark.parametrize("shapes", [[(1, T, 2048) for T in (300, 400, 500, 640)],        # a cluster
                                    [(8, 256, 2048), (8, 768, 512), (24, 128, 512), (50, 96, 512)],
                                    [(1, T, 2048) for T in (1024, 3000, 4096, 5000)]])   # a grid    # one pass over several groups
def test_quantizers_of_different_sizes_at_once(shapes):
    jobs, results = [], []
    for i, (G, R, C) in enumerate(shapes):
        x = torch.randn((G, R, C), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").to(torch.bfloat16)
        want, stream = mxq.quantize_nvfp4(x), torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = {k: torch.zeros_like(v) for k, v in want.items() if torch.is_tensor(v)}
            ws, _ = mxq._workspace("quantize_nvfp4", G, R, C, x.device)
        torch.cuda.synchronize()

        def job(x=x, G=G, R=R, C=C, o=got, ws=ws, stream=stream):
            mxq.mxq_quantize_nvfp4(x, G, R, C, "four_six", "linear", o["codes"], o["scales"], o["s2"], o["mbits"], o["m4_count"],
                                   o["status"], ws, stream=stream)
        jobs.append(job)
        results.append((got, want))
    _together(jobs, 3000)
    for got, want in results:
        assert int(got["status"].item()) == 0
        assert all(torch.equal(got[k], want[k]) for k in ("codes", "scales", "s2"))

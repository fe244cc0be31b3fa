"""The layer operators' refusals, without a GPU: status codes of the C ABI
(every call fails its checks before any launch) and the binding's checks of
types, shapes, sizes and devices (the compute entry points are replaced by a
recorder; host tensors stand in for device tensors)."""
import ctypes

import pytest
import torch

from mxfp_block_scaled_b200 import layers, mxq

OK, ARG, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 6
P = 0x1000                  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return mxq.load()


def call(fn, spec, over):
    args = dict(spec)
    assert set(over) <= set(args)
    args.update(over)
    return fn(*args.values())


QUANT = dict(x=P, rows=4, cols=128, brows=1, bcols=128, codes=P, scales=P, status=P, stream=None)
GEMM = dict(a=P, sa=P, b=P, sb=P, M=4, N=8, K=128, out=0, c=P, status=P, stream=None)
MOE = dict(x=P, T=2, hidden=128, ids=P, w=P, topk=2, fmt=0, experts=4, inter=128, gc=P, gs=P, g2=P, dc=P, ds=P, d2=P,
           y=P, status=P, ws=P, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), ARG), (dict(cols=-16), ARG), (dict(cols=24), SHAPE), (dict(brows=64), UNSUPPORTED),
    (dict(bcols=64), UNSUPPORTED), (dict(brows=0), ARG), (dict(x=None), ARG), (dict(codes=None), ARG),
    (dict(scales=None), ARG), (dict(status=None), ARG), (dict(x=P + 2), ALIGN), (dict(codes=P + 4), ALIGN),
    (dict(scales=P + 2), ALIGN), (dict(status=P + 1), ALIGN), (dict(rows=1 << 40, cols=1 << 40), SHAPE),
    (dict(rows=0, x=None, codes=None, scales=None), OK), (dict(cols=0, x=None, codes=None), OK)])
def test_quantizer_status_codes(lib, over, code):
    assert call(lib.mxq_quantize_fp8, QUANT, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), ARG), (dict(N=-1), ARG), (dict(K=-16), ARG), (dict(K=8), SHAPE), (dict(K=130), SHAPE),
    (dict(out=2), ARG), (dict(a=None), ARG), (dict(sa=None), ARG), (dict(b=None), ARG), (dict(sb=None), ARG),
    (dict(c=None), ARG), (dict(status=None), ARG), (dict(a=P + 8), ALIGN), (dict(b=P + 8), ALIGN),
    (dict(c=P + 8), ALIGN), (dict(sa=P + 2), ALIGN), (dict(sb=P + 1), ALIGN), (dict(status=P + 2), ALIGN),
    (dict(M=1 << 31), SHAPE), (dict(N=1 << 31), SHAPE), (dict(K=1 << 31), SHAPE),
    (dict(M=1 << 30, N=1 << 30), SHAPE), (dict(M=0, a=None, c=None), OK), (dict(N=0, b=None, c=None), OK)])
def test_product_status_codes(lib, over, code):
    assert call(lib.mxq_gemm_fp8, GEMM, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), ARG), (dict(topk=-1), ARG), (dict(hidden=-128), ARG), (dict(experts=0), ARG), (dict(fmt=4), ARG),
    (dict(fmt=-1), ARG), (dict(hidden=64), SHAPE), (dict(inter=192), SHAPE), (dict(hidden=8320), UNSUPPORTED),
    (dict(inter=8320), UNSUPPORTED), (dict(T=1025), UNSUPPORTED), (dict(T=2049, topk=0), UNSUPPORTED),
    (dict(T=1 << 40, topk=1 << 40), UNSUPPORTED), (dict(experts=4097), UNSUPPORTED), (dict(x=None), ARG),
    (dict(ids=None), ARG), (dict(w=None), ARG), (dict(gc=None), ARG), (dict(ds=None), ARG), (dict(g2=None), ARG),
    (dict(d2=None), ARG), (dict(y=None), ARG), (dict(status=None), ARG), (dict(x=P + 8), ALIGN),
    (dict(ids=P + 2), ALIGN), (dict(w=P + 1), ALIGN), (dict(gc=P + 4), ALIGN), (dict(gs=P + 4), ALIGN),
    (dict(dc=P + 8), ALIGN), (dict(ds=P + 8), ALIGN), (dict(g2=P + 2), ALIGN), (dict(y=P + 8), ALIGN),
    (dict(ws=P + 16), ALIGN), (dict(ws=None), WORKSPACE), (dict(wsb=2 * 4 * 128 * 4 - 1), WORKSPACE),
    (dict(T=0, x=None, y=None), OK), (dict(hidden=0, x=None, y=None), OK)])
def test_layer_status_codes(lib, over, code):
    assert call(lib.mxq_moe_forward, MOE, over) == code


def test_layer_workspace_sizes(lib):
    f = lib.mxq_moe_workspace_bytes
    assert f(2, 2, 128, 128) == 2 * 4 * 128 * 4 and f(1, 1, 2048, 768) == (2048 + 768) * 4
    assert f(2048, 1, 8192, 8192) == 2 * 2048 * 8192 * 4 and f(0, 8, 128, 128) == 0
    assert f(2049, 1, 128, 128) == 0 and f(1, 1, 100, 128) == 0 and f(-1, 1, 128, 128) == 0


class _Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name == "mxq_moe_workspace_bytes":
            return self.real.mxq_moe_workspace_bytes

        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def rec(monkeypatch, lib):
    r = _Recorder(lib)
    monkeypatch.setattr(mxq, "load", lambda *a, **k: r)
    monkeypatch.setattr(mxq, "_device", lambda t: t.get_device())
    monkeypatch.setattr(mxq, "_enqueue", lambda fn, args, dev, stream: fn(*args))
    return r


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def stack(fmt, E=3, H=256, I=128):
    def one(R, C):
        q = {"codes": u8(E, R, C if fmt in ("mxfp8", "fp8_block") else C // 2), "fmt": fmt}
        q["scales"] = torch.zeros((E, R // 128, C // 128)) if fmt == "fp8_block" else u8(E, R, C // (16 if fmt == "nvfp4" else 32))
        if fmt == "nvfp4":
            q["s2"] = torch.zeros(E)
        return q
    return {"gate_up": one(2 * I, H), "down": one(H, I)}


def tokens(T=4, k=2, H=256):
    return bf16(T, H), torch.zeros((T, k), dtype=torch.int32), torch.zeros((T, k))


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="device tensors"):
        mxq.mxq_quantize_fp8(bf16(1, 128), 1, 128, 1, 128, u8(128), torch.zeros(1), torch.zeros(1))


def test_wrappers_and_layer_paths_pass_the_checks(rec):
    x, ids, w = tokens()
    for fmt in ("nvfp4", "mxfp4", "mxfp8", "fp8_block"):
        layers.routed_forward(stack(fmt), x, ids, w)
    layers.routed_forward(stack("nvfp4"), x, ids, w, workspace=mxq.moe_workspace(4, 2, 256, 128, "cpu"))
    layers.routed_forward(stack("nvfp4"), x[:0], ids[:0], w[:0])
    wq = mxq.quantize_fp8(bf16(200, 256), 128)
    assert tuple(wq["scales"].shape) == (2, 2)
    layers.fp8_linear(x, wq)
    assert layers.fp8_linear(x, wq, out="f32")["c"].dtype == torch.float32
    q = layers.block_fp8_layer(bf16(3, 256, 128), bf16(3, 128, 128))
    assert tuple(q["gate_up"]["scales"].shape) == (3, 2, 1) and q["down"]["fmt"] == "fp8_block"
    names = [c[0] for c in rec.calls]
    assert (names.count("mxq_moe_forward"), names.count("mxq_gemm_fp8"), names.count("mxq_quantize_fp8")) == (6, 2, 5)
    # the tile's status word goes to both of its steps
    a, b = [c[1] for c in rec.calls if c[0] in ("mxq_quantize_fp8", "mxq_gemm_fp8")][1:3]
    assert a[-1] == b[-1]


def test_wrong_types_shapes_and_strides_are_refused(rec):
    x, ids, w = tokens()
    for fmt in ("nvfp4", "fp8_block"):
        for change in (lambda L: L["gate_up"].update(codes=u8(3, 256, 96)), lambda L: L["down"].update(scales=u8(3, 8, 8)),
                       lambda L: L["down"].update(codes=L["down"]["codes"].float()),
                       lambda L: L["gate_up"].update(codes=L["gate_up"]["codes"].transpose(0, 1).contiguous().transpose(0, 1)),
                       lambda L: L["down"].update(fmt="mxfp8"), lambda L: [L[k].update(fmt="fp8") for k in L]):
            L = stack(fmt)
            change(L)
            with pytest.raises(ValueError):
                layers.routed_forward(L, x, ids, w)
    L = stack("nvfp4")
    for bad in ((x.float(), ids, w), (x, ids.long(), w), (x, ids, w.double()), (x, ids[:3], w), (x, ids, w[:, :1]),
                (x.t().contiguous().t(), ids, w), (x[:, :128].contiguous(), ids, w)):
        with pytest.raises(ValueError):
            layers.routed_forward(L, *bad)
    L["down"]["s2"] = torch.zeros(2)
    with pytest.raises(ValueError, match="s2"):
        layers.routed_forward(L, x, ids, w)
    with pytest.raises(ValueError, match="stack"):
        layers.block_fp8_layer(bf16(3, 200, 128), bf16(3, 128, 100))
    for a in ((u8(2, 128), torch.zeros(2, 2), u8(8, 128), torch.zeros(1, 1)),
              (u8(2, 128), torch.zeros(2, 1), u8(8, 144), torch.zeros(1, 2)),
              (u8(2, 128), torch.zeros(2, 1), u8(129, 128), torch.zeros(1, 1)),
              (u8(2, 128).float(), torch.zeros(2, 1), u8(8, 128), torch.zeros(1, 1)),
              (u8(128, 2).t(), torch.zeros(2, 1), u8(8, 128), torch.zeros(1, 1))):
        with pytest.raises(ValueError):
            mxq.gemm_fp8(*a)
    ok = (u8(2, 128), torch.zeros(2, 1), u8(8, 128), torch.zeros(1, 1))
    with pytest.raises(ValueError, match="out is one of"):
        mxq.gemm_fp8(*ok, out="f16")
    with pytest.raises(ValueError, match="128 x 128"):
        mxq.quantize_fp8(bf16(4, 128), brows=32)
    assert not rec.calls


@pytest.mark.parametrize("short", ["a", "sa", "b", "sb", "c", "status"])
def test_product_buffers_smaller_than_the_call_are_refused(rec, short):
    t = dict(a=u8(5 * 144), sa=torch.zeros(10), b=u8(130 * 144), sb=torch.zeros(4), c=bf16(650),
             status=torch.zeros(1, dtype=torch.int32))
    mxq.mxq_gemm_fp8(t["a"], t["sa"], t["b"], t["sb"], 5, 130, 144, "bf16", t["c"], t["status"])
    t[short] = t[short][:-1]
    with pytest.raises(ValueError, match="the call needs"):
        mxq.mxq_gemm_fp8(t["a"], t["sa"], t["b"], t["sb"], 5, 130, 144, "bf16", t["c"], t["status"])
    assert len(rec.calls) == 1


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8", "fp8_block"])
def test_layer_buffers_smaller_than_the_call_are_refused(rec, fmt):
    E, H, I, T, k = 3, 256, 128, 4, 2
    L = stack(fmt)
    x, ids, w = tokens()
    names = ("x", "ids", "w", "gc", "gs", "g2", "dc", "ds", "d2", "y", "status")
    full = dict(zip(names, (x, ids, w, L["gate_up"]["codes"], L["gate_up"]["scales"], L["gate_up"].get("s2"),
                            L["down"]["codes"], L["down"]["scales"], L["down"].get("s2"), bf16(T, H),
                            torch.zeros(1, dtype=torch.int32))))
    ws = mxq.moe_workspace(T, k, H, I, "cpu")

    def go(t):
        mxq.mxq_moe_forward(t["x"], T, H, t["ids"], t["w"], k, fmt, E, I, t["gc"], t["gs"], t["g2"], t["dc"], t["ds"],
                            t["d2"], t["y"], t["status"], ws)
    go(full)
    for n in names:
        if full[n] is not None:
            with pytest.raises(ValueError, match="the call needs"):
                go(dict(full, **{n: full[n].reshape(-1)[:-1]}))
            if full[n].numel() > 1:
                with pytest.raises(ValueError, match="contiguous"):
                    go(dict(full, **{n: torch.stack((full[n], full[n]), -1)[..., 0]}))
    assert len(rec.calls) == 1


def test_quantizer_buffers_smaller_than_the_call_are_refused(rec):
    x, codes, scales, st = bf16(130, 144), u8(130, 144), torch.zeros(260), torch.zeros(1, dtype=torch.int32)
    mxq.mxq_quantize_fp8(x, 130, 144, 1, 128, codes, scales, st)
    mxq.mxq_quantize_fp8(x, 130, 144, 128, 128, codes, scales[:4], st)
    for bad in ((x[:-1], codes, scales, st), (x, codes[:-1], scales, st), (x, codes, scales[:-1], st)):
        with pytest.raises(ValueError, match="the call needs"):
            mxq.mxq_quantize_fp8(bad[0], 130, 144, 1, 128, *bad[1:])
    assert len(rec.calls) == 2


def test_buffers_on_different_devices_are_refused(rec, monkeypatch):
    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 1
    x, codes, scales = bf16(2, 128), u8(2, 128), torch.zeros(2)
    st = torch.zeros(1, dtype=torch.int32).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="not on the device"):
        mxq.mxq_quantize_fp8(x, 2, 128, 1, 128, codes, scales, st)
    assert not rec.calls


def test_enumerators_match_the_header():
    text = open(mxq.__file__.rsplit("/", 2)[0] + "/include/mxq.h").read()
    assert "MXQ_FMT_FP8_BLOCK = %d" % mxq.FMT["fp8_block"] in text
    assert "MXQ_OUT_BF16 = %d" % mxq.OUT["bf16"] in text and "MXQ_OUT_F32 = %d" % mxq.OUT["f32"] in text
    assert isinstance(ctypes.c_uint32(mxq.DEV_INVALID_EXPERT).value, int)

"""Refusals of the linear and cache operators, without a GPU: status codes of the C
ABI (every call fails its checks before any launch) and the binding's checks of types,
shapes, sizes and devices (the compute entry points are replaced by a recorder; host
tensors stand in for device tensors)."""
import ctypes

import pytest
import torch

from mxfp_block_scaled_b200 import layers, mxq

OK, ARG, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 6
P = 0x1000                  # never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return mxq.load()


def call(fn, spec, over):
    args = dict(spec)
    assert set(over) <= set(args)
    args.update(over)
    return fn(*args.values())


LINEAR = dict(x=P, T=2, K=64, fmt=0, codes=P, scales=P, s2=P, N=8, out=0, y=P, status=P, ws=P, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), ARG), (dict(N=-1), ARG), (dict(K=-32), ARG), (dict(out=2), ARG), (dict(fmt=3), ARG), (dict(fmt=-1), ARG),
    (dict(K=48), SHAPE), (dict(N=1 << 31), SHAPE), (dict(T=2049), UNSUPPORTED), (dict(K=65568), UNSUPPORTED),
    (dict(x=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(s2=None), ARG), (dict(y=None), ARG),
    (dict(status=None), ARG), (dict(x=P + 8), ALIGN), (dict(codes=P + 8), ALIGN), (dict(s2=P + 2), ALIGN),
    (dict(y=P + 1), ALIGN), (dict(out=1, y=P + 2), ALIGN), (dict(status=P + 2), ALIGN), (dict(ws=P + 16), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE), (dict(T=0, x=None, y=None), OK),
    (dict(N=0, codes=None, y=None), OK)])
def test_linear_status_codes(lib, over, code):
    assert call(lib.mxq_linear, LINEAR, over) == code


def test_linear_workspace_sizes(lib):
    f = lib.mxq_linear_workspace_bytes
    assert f(1, 2048) >= 2048 * 2 + 4 and f(2048, 65536) >= 2048 * 65536 * 2
    assert f(0, 64) == 0 and f(-1, 64) == 0 and f(1, 48) == 0 and f(2049, 64) == 0 and f(1, 65568) == 0


def struct(**over):
    a = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, k_s2=P, v_s2=P, pages=4, kv_heads=2, page_tokens=16,
             head_dim=64, fmt=0)
    assert set(over) <= set(a)
    a.update(over)
    return ctypes.byref(mxq._CacheStruct(*a.values()))


WRITE = dict(cache=None, k=P, ks=128, v=P, vs=128, T=2, cu=P, lens=P, table=P, seqs=1, width=1, mode=0, status=P, stream=None)
READ = dict(cache=None, cu=P, lens=P, table=P, seqs=1, width=1, T=2, k=P, v=P, status=P, stream=None)
ATT = dict(cache=None, q=P, qs=256, T=2, heads=4, cu=P, lens=P, table=P, seqs=1, width=1, max_new=2, scale=1.0, o=P, lse=P,
           status=P, ws=P, wsb=1 << 30, stream=None)
CALLS = [("mxq_cache_write", WRITE), ("mxq_cache_read", READ), ("mxq_cache_attention", ATT)]


@pytest.mark.parametrize("name,spec", CALLS)
@pytest.mark.parametrize("over,code", [
    (dict(pages=-1), ARG), (dict(kv_heads=0), ARG), (dict(page_tokens=0), ARG), (dict(head_dim=0), ARG), (dict(fmt=9), ARG),
    (dict(fmt=1), UNSUPPORTED), (dict(fmt=3), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED),
    (dict(page_tokens=24), UNSUPPORTED), (dict(page_tokens=512), UNSUPPORTED), (dict(pages=1 << 31), SHAPE),
    (dict(k_codes=None), ARG), (dict(v_scales=None), ARG), (dict(k_s2=None), ARG), (dict(v_codes=P + 8), ALIGN),
    (dict(k_scales=P + 8), ALIGN), (dict(v_s2=P + 2), ALIGN)])
def test_caches_that_every_call_refuses(lib, name, spec, over, code):
    assert call(getattr(lib, name), spec, dict(cache=struct(**over))) == code


@pytest.mark.parametrize("name,spec", CALLS)
@pytest.mark.parametrize("over,code", [
    (dict(T=-1), ARG), (dict(seqs=-1), ARG), (dict(width=-1), ARG), (dict(cache=None), ARG), (dict(cu=None), ARG),
    (dict(lens=None), ARG), (dict(table=None), ARG), (dict(status=None), ARG), (dict(cu=P + 2), ALIGN),
    (dict(lens=P + 1), ALIGN), (dict(table=P + 2), ALIGN), (dict(status=P + 2), ALIGN), (dict(T=1 << 31), SHAPE),
    (dict(width=1 << 31), SHAPE), (dict(seqs=4097), UNSUPPORTED), (dict(T=0), OK), (dict(seqs=0), OK)])
def test_batches_that_every_call_refuses(lib, name, spec, over, code):
    assert call(getattr(lib, name), spec, dict(dict(cache=struct()), **over)) == code


@pytest.mark.parametrize("name,spec,over,code", [
    ("mxq_cache_write", WRITE, dict(mode=7), ARG), ("mxq_cache_write", WRITE, dict(ks=120), SHAPE),
    ("mxq_cache_write", WRITE, dict(vs=132), ALIGN), ("mxq_cache_write", WRITE, dict(vs=1 << 40), SHAPE),
    ("mxq_cache_write", WRITE, dict(k=None), ARG), ("mxq_cache_write", WRITE, dict(v=P + 8), ALIGN),
    ("mxq_cache_read", READ, dict(k=None), ARG), ("mxq_cache_read", READ, dict(v=P + 8), ALIGN),
    ("mxq_cache_attention", ATT, dict(heads=0), ARG), ("mxq_cache_attention", ATT, dict(heads=3), SHAPE),
    ("mxq_cache_attention", ATT, dict(heads=2 * 257, qs=1 << 16), UNSUPPORTED),
    ("mxq_cache_attention", ATT, dict(T=1 << 29), SHAPE), ("mxq_cache_attention", ATT, dict(T=(1 << 31) - 1, heads=512, qs=1 << 15), SHAPE),
    ("mxq_cache_attention", ATT, dict(max_new=-1), ARG), ("mxq_cache_attention", ATT, dict(qs=248), SHAPE),
    ("mxq_cache_attention", ATT, dict(qs=260), ALIGN), ("mxq_cache_attention", ATT, dict(scale=NAN), ARG),
    ("mxq_cache_attention", ATT, dict(scale=INF), ARG), ("mxq_cache_attention", ATT, dict(q=None), ARG),
    ("mxq_cache_attention", ATT, dict(o=None), ARG), ("mxq_cache_attention", ATT, dict(o=P + 8), ALIGN),
    ("mxq_cache_attention", ATT, dict(lse=P + 2), ALIGN), ("mxq_cache_attention", ATT, dict(ws=None), WORKSPACE),
    ("mxq_cache_attention", ATT, dict(wsb=64), WORKSPACE), ("mxq_cache_attention", ATT, dict(ws=P + 16), ALIGN)])
def test_cache_status_codes(lib, name, spec, over, code):
    assert call(getattr(lib, name), spec, dict(dict(cache=struct()), **over)) == code


def test_attention_workspace_sizes(lib):
    f = lib.mxq_cache_attention_workspace_bytes
    assert f(struct(), 2, 4, 1, 1) > 0 and f(struct(), 2, 3, 1, 1) == 0 and f(struct(fmt=1), 2, 4, 1, 1) == 0
    # wider heads and more rows a sequence take no less
    assert f(struct(head_dim=128), 2, 4, 1, 1) >= f(struct(), 2, 4, 1, 1)
    assert f(struct(), 4096, 4, 1, 4096) >= f(struct(), 4096, 4, 1, 1)


# ------------------------------------------------------------- binding --
class _Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def rec(monkeypatch, lib):
    r = _Recorder(lib)
    monkeypatch.setattr(mxq, "load", lambda *a, **k: r)
    monkeypatch.setattr(mxq, "_device", lambda t: t.get_device())
    monkeypatch.setattr(mxq, "_cache_device", lambda c: c.k_codes.get_device())
    monkeypatch.setattr(mxq, "_enqueue", lambda fn, args, dev, stream: fn(*args))
    return r


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def a_cache(fmt="mxfp8", pages=4, heads=2, tokens=16, dim=64):
    s2 = (torch.ones(heads), torch.ones(heads)) if fmt == "nvfp4" else (None, None)
    return mxq.Cache.empty(pages, heads, tokens, dim, fmt, *s2, device="cpu")


def a_batch(B=2, width=2):
    return torch.arange(B + 1, dtype=torch.int32) * 2, torch.full((B,), 9, dtype=torch.int32), torch.zeros((B, width), dtype=torch.int32)


def test_host_tensors_are_refused():
    cache, st, b = a_cache(), i32(0), a_batch()
    with pytest.raises(ValueError, match="device tensors"):
        mxq.mxq_linear(bf16(1, 64), 1, 64, "mxfp8", u8(8, 64), u8(8, 2), None, 8, "bf16", bf16(1, 8), st, u8(4096))
    with pytest.raises(ValueError, match="device tensors"):
        mxq.mxq_cache_write(cache, bf16(4, 128), 128, bf16(4, 128), 128, 4, *b, 2, 2, "rtn", st)
    with pytest.raises(ValueError, match="device tensors"):
        mxq.mxq_cache_read(cache, *b, 2, 2, 4, bf16(4, 128), bf16(4, 128), st)
    with pytest.raises(ValueError, match="device tensors"):
        mxq.mxq_cache_attention(cache, bf16(4, 256), 256, 4, 4, *b, 2, 2, 2, 1.0, bf16(4, 256), None, st, u8(1 << 20))


def test_wrappers_and_layer_paths_pass_the_checks(rec):
    b = a_batch()
    for fmt in ("mxfp8", "nvfp4"):
        cache = a_cache(fmt)
        qkv = bf16(4, 8, 64)                # four query heads, two of keys, two of values
        out = layers.attention_forward(cache, qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], *b, 2)
        assert tuple(out["o"].shape) == (4, 4, 64) and tuple(out["lse"].shape) == (4, 4)
        (_, w), (_, a) = rec.calls[-2:]
        assert w[2] == w[4] == a[2] == 512 and a[-3] == w[-1] == out["status"].data_ptr()
        assert tuple(mxq.cache_read(cache, *b, 4)["k"].shape) == (4, 2, 64)
        mxq.cache_attention(cache, qkv[:, :4], *b, 2, scale=0.5,
                            workspace=mxq.cache_attention_workspace(cache, 4, 4, 2, 2))
    for q in (dict(codes=u8(24, 128), scales=u8(24, 16), s2=torch.zeros(1), fmt="nvfp4"),
              dict(codes=u8(24, 128), scales=u8(24, 8), fmt="mxfp4"), dict(codes=u8(24, 256), scales=u8(24, 8), fmt="mxfp8"),
              layers.quantize_projection(bf16(24, 256), "fp8_block")):
        r = layers.projection_forward(q, bf16(3, 256), out="f32")
        assert tuple(r["y"].shape) == (3, 24) and r["y"].dtype == torch.float32
    w = {"codes": u8(24, 64), "scales": u8(24, 2)}
    assert mxq.linear(bf16(3, 64), w, "mxfp8", workspace=mxq.linear_workspace(3, 64, "cpu"))["y"].dtype == torch.bfloat16


def test_wrong_types_shapes_and_strides_are_refused(rec):
    cache, (cu, lens, table) = a_cache(), a_batch()
    k, q = bf16(4, 2, 64), bf16(4, 4, 64)
    for a in ((k.float(), k), (k, k[:3]), (bf16(4, 2, 32), k), (bf16(4, 1, 64), k), (k.transpose(1, 2).contiguous().transpose(1, 2), k),
              (bf16(4, 4, 64)[:, ::2], k)):
        with pytest.raises(ValueError):
            mxq.cache_write(cache, *a, cu, lens, table)
    for bad in ((cu.long(), lens, table), (cu[:2], lens, table), (cu, lens.float(), table), (cu, lens, table[:1]),
                (cu, lens, table.t().contiguous().t()), (cu, lens, table[0]), (cu, lens[:, None], table)):
        with pytest.raises(ValueError):
            mxq.cache_write(cache, k, k, *bad)
        with pytest.raises(ValueError):
            mxq.cache_read(cache, *bad, 4)
        with pytest.raises(ValueError):
            mxq.cache_attention(cache, q, *bad, 2)
    for bad in (q[0], q.float(), bf16(4, 4, 32)):
        with pytest.raises(ValueError):
            mxq.cache_attention(cache, bad, cu, lens, table, 2)
    with pytest.raises(KeyError):
        mxq.cache_write(cache, k, k, cu, lens, table, mode="nearest")
    x, w = bf16(3, 64), {"codes": u8(24, 64), "scales": u8(24, 2)}
    for bad in ((x.float(), w, "mxfp8"), (x, w, "mxfp4"), (x, dict(w, scales=u8(24, 4)), "mxfp8"), (x, w, "fp8"),
                (bf16(64, 3).t(), w, "mxfp8"), (x, {"codes": u8(24, 32), "scales": u8(24, 4), "s2": torch.zeros(2)}, "nvfp4")):
        with pytest.raises(ValueError):
            mxq.linear(*bad)
    with pytest.raises(ValueError, match="out is one of"):
        mxq.linear(x, w, "mxfp8", out="f16")
    assert not rec.calls


@pytest.mark.parametrize("bad", [
    dict(fmt="mxfp4"), dict(k_codes=u8(4, 2, 16, 96)), dict(k_codes=u8(4, 2, 16)), dict(v_codes=u8(4, 2, 16, 128)),
    dict(k_scales=u8(4, 2, 16, 4)), dict(v_scales=torch.zeros(4, 2, 16, 2)), dict(v_codes=u8(4, 2, 64, 16).transpose(2, 3)),
    dict(k_codes=u8(4, 2, 24, 64)), dict(fmt="nvfp4")])
def test_caches_of_wrong_tensors_are_refused(bad):
    t = dict(k_codes=u8(4, 2, 16, 64), k_scales=u8(4, 2, 16, 2), v_codes=u8(4, 2, 16, 64), v_scales=u8(4, 2, 16, 2), fmt="mxfp8")
    mxq.Cache(**t)
    with pytest.raises(ValueError):
        mxq.Cache(**dict(t, **bad))
    good = dict(k_codes=u8(4, 2, 16, 32), k_scales=u8(4, 2, 16, 4), v_codes=u8(4, 2, 16, 32), v_scales=u8(4, 2, 16, 4),
                fmt="nvfp4", k_s2=torch.ones(2), v_s2=torch.ones(2))
    mxq.Cache(**good)
    for s2 in (None, torch.ones(3), torch.ones(2).double()):
        with pytest.raises(ValueError):
            mxq.Cache(**dict(good, v_s2=s2))


@pytest.mark.parametrize("short", ["x", "codes", "scales", "s2", "y", "status"])
def test_linear_buffers_smaller_than_the_call_are_refused(rec, short):
    t = dict(x=bf16(3 * 64), codes=u8(24 * 32), scales=u8(24 * 4), s2=torch.zeros(1), y=bf16(72), status=i32(0))

    def go():
        mxq.mxq_linear(t["x"], 3, 64, "nvfp4", t["codes"], t["scales"], t["s2"], 24, "bf16", t["y"], t["status"], u8(4096))
    go()
    t[short] = t[short][:-1]
    with pytest.raises(ValueError, match="the call needs"):
        go()
    assert len(rec.calls) == 1


@pytest.mark.parametrize("short", ["cu", "lens", "table", "k", "v", "o", "lse", "status", "q"])
def test_cache_buffers_smaller_than_the_call_are_refused(rec, short):
    cache = a_cache()
    t = dict(zip(("cu", "lens", "table"), a_batch()), k=bf16(3 * 200 + 128), v=bf16(512), o=bf16(4 * 256), lse=torch.zeros(16),
             status=i32(0), q=bf16(3 * 264 + 256))
    t["table"] = t["table"].reshape(-1)

    def go():
        b = t["cu"], t["lens"], t["table"], 2, 2
        mxq.mxq_cache_write(cache, t["k"], 200, t["v"], 128, 4, *b, "rtn", t["status"])
        mxq.mxq_cache_read(cache, *b, 4, bf16(512), t["v"], t["status"])
        mxq.mxq_cache_attention(cache, t["q"], 264, 4, 4, *b, 2, 1.0, t["o"], t["lse"], t["status"], u8(1 << 20))
    go()
    t[short] = t[short][:-1].clone()
    with pytest.raises(ValueError, match="the call needs|does not hold"):
        go()

"""Thin Python binding of libmxq.so (include/mxq.h).

Argument marshalling only: every step of the quantizer and the verifier
runs in the CUDA library.  Torch provides device memory and the current
CUDA stream; tensors are passed by data pointer.  There is no fallback: if
the library is missing the first call raises.

Low-level functions carry the C names (``mxq_quantize_nvfp4`` ...) and take
tensors for every buffer.  ``quantize_nvfp4``, ``quantize_mx``,
``quantize_act`` and ``dequant_relerr`` allocate the outputs and workspace
with torch and return them.
"""
import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxq.so")

MXQ_OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "shape", 3: "align", 4: "workspace",
                5: "cuda", 6: "unsupported"}
DEV_NONFINITE_INPUT = 0x1
DEV_WAIT_TIMEOUT = 0x2
DEV_INVALID_SCALE = 0x4
DEV_INVALID_EXPERT = 0x8
DEV_INVALID_PAGE = 0x10

FMT = {"nvfp4": 0, "mxfp4": 1, "mxfp8": 2, "fp8_block": 3}
SCALE_MODE = {"rtn": 0, "four_six": 1}
LAYOUT = {"linear": 0, "swizzled_128x4": 1}
OUT = {"bf16": 0, "f32": 1}
OP = {"quantize_nvfp4": 0, "quantize_act": 1, "dequant_relerr": 2}

EXPORTED = ("mxq_version", "mxq_status_string", "mxq_scale_bytes", "mxq_workspace_bytes",
            "mxq_quantize_nvfp4", "mxq_global_scale_nvfp4", "mxq_quantize_nvfp4_s2", "mxq_quantize_nvfp4_weighted",
            "mxq_quantize_mx", "mxq_requant_fp8_mx", "mxq_quantize_act", "mxq_dequant_relerr",
            "mxq_dequant_relerr_noalloc", "mxq_census_reset", "mxq_census_add", "mxq_quantize_fp8",
            "mxq_gemm_fp8", "mxq_moe_workspace_bytes", "mxq_moe_forward", "mxq_linear_workspace_bytes", "mxq_linear",
            "mxq_cache_write", "mxq_cache_read", "mxq_cache_attention_workspace_bytes", "mxq_cache_attention")

# Fields of struct mxq_census (include/mxq.h), in order, each 8 bytes.
CENSUS_FIELDS = ("sum_relerr", "max_relerr", "sum_sq_err", "sum_sq_ref", "sum_sq_err_rtn",
                 "n_tensors", "n_tensors_rtn", "blocks", "blocks_m4",
                 "mean_relerr", "sse_vs_rtn", "m4_fraction", "reserved")
_CENSUS_INTS = ("n_tensors", "n_tensors_rtn", "blocks", "blocks_m4")


class _CacheStruct(ctypes.Structure):
    """struct mxq_cache (include/mxq.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_s2", "v_s2")]
                + [(n, ctypes.c_int64) for n in ("pages", "kv_heads", "page_tokens", "head_dim")]
                + [("fmt", ctypes.c_int)])


class MxqError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__("%s failed: %s (%d)" % (fn, STATUS_NAMES.get(code, "?"), code))
        self.code = code


_lib = None


def load(path=LIB_PATH):
    """Load libmxq.so and declare its signatures (raises if missing)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libmxq.so is not built (%s): run `python -m mxfp_block_scaled_b200.build`"
                           % path)
    L = ctypes.CDLL(path)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.mxq_version.restype = i32
    L.mxq_version.argtypes = []
    L.mxq_status_string.restype = ctypes.c_char_p
    L.mxq_status_string.argtypes = [i32]
    L.mxq_scale_bytes.restype = sz
    L.mxq_scale_bytes.argtypes = [i32, i32, i64, i64, i64]
    L.mxq_workspace_bytes.restype = sz
    L.mxq_workspace_bytes.argtypes = [i32, i64, i64, i64]
    L.mxq_quantize_nvfp4.restype = i32
    L.mxq_quantize_nvfp4.argtypes = [vp, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.mxq_global_scale_nvfp4.restype = i32
    L.mxq_global_scale_nvfp4.argtypes = [vp, i64, i64, i64, vp, vp, vp]
    L.mxq_quantize_nvfp4_s2.restype = i32
    L.mxq_quantize_nvfp4_s2.argtypes = [vp, i64, i64, i64, vp, i32, i32, vp, vp, vp, vp, vp, vp]
    L.mxq_census_reset.restype = i32
    L.mxq_census_reset.argtypes = [vp, vp]
    L.mxq_census_add.restype = i32
    L.mxq_census_add.argtypes = [vp, i64, vp, vp, vp, vp, i64, vp, i64, vp]
    L.mxq_quantize_nvfp4_weighted.restype = i32
    L.mxq_quantize_nvfp4_weighted.argtypes = [vp, i64, i64, i64, vp, i64, i32, vp, vp, vp, vp, vp, sz,
                                              vp]
    L.mxq_quantize_mx.restype = i32
    L.mxq_quantize_mx.argtypes = [vp, i64, i64, i32, i32, i32, vp, vp, vp, vp]
    L.mxq_requant_fp8_mx.restype = i32
    L.mxq_requant_fp8_mx.argtypes = [vp, vp, i64, i64, i64, i64, i32, i32, vp, vp, vp, vp]
    L.mxq_quantize_act.restype = i32
    L.mxq_quantize_act.argtypes = [vp, i64, i64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.mxq_dequant_relerr.restype = i32
    L.mxq_dequant_relerr.argtypes = [vp, vp, vp, vp, i32, i32, i64, i64, i64, i64, vp, vp, vp, vp, sz,
                                     vp]
    L.mxq_dequant_relerr_noalloc.restype = i32
    L.mxq_dequant_relerr_noalloc.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, i64, vp, vp, vp, vp]
    L.mxq_quantize_fp8.restype = i32
    L.mxq_quantize_fp8.argtypes = [vp, i64, i64, i64, i64, vp, vp, vp, vp]
    L.mxq_gemm_fp8.restype = i32
    L.mxq_gemm_fp8.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, vp, vp]
    L.mxq_moe_workspace_bytes.restype = sz
    L.mxq_moe_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.mxq_moe_forward.restype = i32
    L.mxq_moe_forward.argtypes = [vp, i64, i64, vp, vp, i64, i32, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                  vp, sz, vp]
    cp = ctypes.POINTER(_CacheStruct)
    L.mxq_linear_workspace_bytes.restype = sz
    L.mxq_linear_workspace_bytes.argtypes = [i64, i64]
    L.mxq_linear.restype = i32
    L.mxq_linear.argtypes = [vp, i64, i64, i32, vp, vp, vp, i64, i32, vp, vp, vp, sz, vp]
    L.mxq_cache_write.restype = i32
    L.mxq_cache_write.argtypes = [cp, vp, i64, vp, i64, i64, vp, vp, vp, i64, i64, i32, vp, vp]
    L.mxq_cache_read.restype = i32
    L.mxq_cache_read.argtypes = [cp, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp]
    L.mxq_cache_attention_workspace_bytes.restype = sz
    L.mxq_cache_attention_workspace_bytes.argtypes = [cp, i64, i64, i64, i64]
    L.mxq_cache_attention.restype = i32
    L.mxq_cache_attention.argtypes = [cp, vp, i64, i64, i64, vp, vp, vp, i64, i64, i64, ctypes.c_float, vp, vp, vp, vp,
                                      sz, vp]
    L.mxq_test_stall_next_single_pass.restype = None
    L.mxq_test_stall_next_single_pass.argtypes = [i32]
    L.mxq_test_stall_next_product.restype = None
    L.mxq_test_stall_next_product.argtypes = [i32]
    L.mxq_test_stall_next_attention.restype = None
    L.mxq_test_stall_next_attention.argtypes = [i32]
    if path == LIB_PATH:
        _lib = L
    return L


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmxq takes device tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, rc):
    if rc != MXQ_OK:
        raise MxqError(fn, rc)


def scale_bytes(fmt, layout, n_matrices, rows, cols):
    return load().mxq_scale_bytes(FMT[fmt], LAYOUT[layout], n_matrices, rows, cols)


def workspace_bytes(op, n, rows, cols):
    return load().mxq_workspace_bytes(OP[op], n, rows, cols)


def _workspace(op, n, rows, cols, device):
    nbytes = workspace_bytes(op, n, rows, cols)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device), nbytes


def _nbytes(t):
    return 0 if t is None else t.nbytes


def _need(name, t, nbytes):
    """The library sees only a pointer, so a buffer that is not contiguous or
    is smaller than the call reads or writes is refused here, before anything
    is enqueued (the kernels would otherwise touch memory past its end).
    Sizes the library rejects (negative, misaligned shapes) give nbytes <= 0
    here and are left to its status code."""
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if _nbytes(t) < nbytes:
        raise ValueError("%s holds %d bytes; the call needs %d" % (name, _nbytes(t), nbytes))


def _verify_scale_need(fmt, layout, n_tensors, rows, cols, tps):
    """Scale bytes the verifier reads: n_tensors * rows * cols / block when
    linear; tiled, each run of tps tensors is one scale matrix (the last run
    may be shorter)."""
    if layout == "linear" or tps < 1:
        return scale_bytes(fmt, "linear", n_tensors, rows, cols)
    full, rem = divmod(n_tensors, tps)
    return (scale_bytes(fmt, layout, full, rows * tps, cols)
            + (scale_bytes(fmt, layout, 1, rows * rem, cols) if rem else 0))


def _code_bytes(fmt, n):
    return n if fmt == "mxfp8" else n // 2


# ---------------------------------------------------------------- C names --
def mxq_quantize_nvfp4(x, n_groups, rows, cols, mode, layout, codes, scales, s2, mbits, m4_count,
                       status, workspace, stream=None):
    n = n_groups * rows * cols
    _need("x", x, 2 * n)
    _need("codes", codes, n // 2)
    _need("scales", scales, scale_bytes("nvfp4", layout, n_groups, rows, cols))
    _need("s2", s2, 4 * n_groups)
    _need("mbits", mbits, 4 * ((n // 16 + 31) // 32))
    _need("m4_count", m4_count, 4 * n_groups)
    _need("status", status, 4)
    rc = load().mxq_quantize_nvfp4(_p(x), n_groups, rows, cols, SCALE_MODE[mode], LAYOUT[layout],
                                   _p(codes),
                                   _p(scales), _p(s2), _p(mbits), _p(m4_count), _p(status),
                                   _p(workspace), _nbytes(workspace), _stream(stream))
    _check("mxq_quantize_nvfp4", rc)


def mxq_global_scale_nvfp4(x, n_groups, rows, cols, s2, status, stream=None):
    _need("x", x, 2 * n_groups * rows * cols)
    _need("s2", s2, 4 * n_groups)
    _need("status", status, 4)
    rc = load().mxq_global_scale_nvfp4(_p(x), n_groups, rows, cols, _p(s2), _p(status), _stream(stream))
    _check("mxq_global_scale_nvfp4", rc)


def mxq_quantize_nvfp4_s2(x, n_groups, rows, cols, s2_in, mode, layout, codes, scales, mbits, m4_count,
                          status, stream=None):
    n = n_groups * rows * cols
    _need("x", x, 2 * n)
    _need("s2_in", s2_in, 4 * n_groups)
    _need("codes", codes, n // 2)
    _need("scales", scales, scale_bytes("nvfp4", layout, n_groups, rows, cols))
    _need("mbits", mbits, 4 * ((n // 16 + 31) // 32))
    _need("m4_count", m4_count, 4 * n_groups)
    _need("status", status, 4)
    rc = load().mxq_quantize_nvfp4_s2(_p(x), n_groups, rows, cols, _p(s2_in), SCALE_MODE[mode],
                                      LAYOUT[layout], _p(codes), _p(scales), _p(mbits), _p(m4_count),
                                      _p(status), _stream(stream))
    _check("mxq_quantize_nvfp4_s2", rc)


def mxq_census_reset(census, stream=None):
    _need("census", census, 8 * len(CENSUS_FIELDS))
    _check("mxq_census_reset", load().mxq_census_reset(_p(census), _stream(stream)))


def mxq_census_add(census, n_tensors, sum_sq_err, sum_sq_ref, relerr, sum_sq_err_rtn, n_groups,
                   m4_count, blocks_per_group, stream=None):
    _need("census", census, 8 * len(CENSUS_FIELDS))
    for name, t in (("sum_sq_err", sum_sq_err), ("sum_sq_ref", sum_sq_ref), ("relerr", relerr),
                    ("sum_sq_err_rtn", sum_sq_err_rtn)):
        _need(name, t, 8 * n_tensors)
    _need("m4_count", m4_count, 4 * n_groups)
    rc = load().mxq_census_add(_p(census), n_tensors, _p(sum_sq_err), _p(sum_sq_ref), _p(relerr),
                               _p(sum_sq_err_rtn), n_groups, _p(m4_count), blocks_per_group,
                               _stream(stream))
    _check("mxq_census_add", rc)


def mxq_quantize_nvfp4_weighted(x, n_groups, rows, cols, h, h_groups, layout, codes, scales, s2,
                                status, workspace, stream=None):
    n = n_groups * rows * cols
    _need("x", x, 2 * n)
    _need("h", h, 4 * h_groups * cols)
    _need("codes", codes, n // 2)
    _need("scales", scales, scale_bytes("nvfp4", layout, n_groups, rows, cols))
    _need("s2", s2, 4 * n_groups)
    _need("status", status, 4)
    rc = load().mxq_quantize_nvfp4_weighted(_p(x), n_groups, rows, cols, _p(h), h_groups,
                                            LAYOUT[layout], _p(codes), _p(scales), _p(s2), _p(status),
                                            _p(workspace), _nbytes(workspace), _stream(stream))
    _check("mxq_quantize_nvfp4_weighted", rc)


def mxq_quantize_mx(x, rows, cols, fmt, block, layout, codes, scales, status, stream=None):
    n = rows * cols
    _need("x", x, 2 * n)
    _need("codes", codes, _code_bytes(fmt, n))
    _need("scales", scales, scale_bytes(fmt, layout, 1, rows, cols))
    _need("status", status, 4)
    rc = load().mxq_quantize_mx(_p(x), rows, cols, FMT[fmt], block, LAYOUT[layout], _p(codes),
                                _p(scales), _p(status), _stream(stream))
    _check("mxq_quantize_mx", rc)


def mxq_requant_fp8_mx(fp8, bscale, rows, cols, brows, bcols, fmt, layout, codes, scales, status,
                       stream=None):
    n = rows * cols
    _need("fp8", fp8, n)
    if brows > 0 and bcols > 0:
        _need("bscale", bscale, 4 * (-(-rows // brows)) * (-(-cols // bcols)))
    _need("codes", codes, _code_bytes(fmt, n))
    _need("scales", scales, scale_bytes(fmt, layout, 1, rows, cols))
    _need("status", status, 4)
    rc = load().mxq_requant_fp8_mx(_p(fp8), _p(bscale), rows, cols, brows, bcols, FMT[fmt],
                                   LAYOUT[layout], _p(codes), _p(scales), _p(status), _stream(stream))
    _check("mxq_requant_fp8_mx", rc)


def mxq_quantize_act(tokens, T, hidden, fmt, mode, layout, codes, scales, input_scale, status,
                     workspace, stream=None):
    n = T * hidden
    _need("tokens", tokens, 2 * n)
    _need("codes", codes, _code_bytes(fmt, n))
    _need("scales", scales, scale_bytes(fmt, layout, 1, T, hidden))
    _need("input_scale", input_scale, 4 if fmt == "nvfp4" else 0)
    _need("status", status, 4)
    rc = load().mxq_quantize_act(_p(tokens), T, hidden, FMT[fmt], SCALE_MODE[mode], LAYOUT[layout],
                                 _p(codes), _p(scales),
                                 _p(input_scale), _p(status), _p(workspace),
                                 _nbytes(workspace), _stream(stream))
    _check("mxq_quantize_act", rc)


def _need_verify(x, codes, scales, s2, fmt, layout, n_tensors, rows, cols, tps, err, ref, rel):
    n = n_tensors * rows * cols
    _need("x", x, 2 * n)
    _need("codes", codes, _code_bytes(fmt, n))
    _need("scales", scales, _verify_scale_need(fmt, layout, n_tensors, rows, cols, tps))
    if fmt == "nvfp4" and tps >= 1:
        _need("s2", s2, 4 * (-(-n_tensors // tps)))
    for name, t in (("sum_sq_err", err), ("sum_sq_ref", ref), ("relerr", rel)):
        _need(name, t, 8 * n_tensors)


def mxq_dequant_relerr(x, codes, scales, s2, fmt, layout, n_tensors, rows, cols,
                       tensors_per_scale, sum_sq_err, sum_sq_ref, relerr, workspace, stream=None):
    _need_verify(x, codes, scales, s2, fmt, layout, n_tensors, rows, cols, tensors_per_scale,
                 sum_sq_err, sum_sq_ref, relerr)
    rc = load().mxq_dequant_relerr(_p(x), _p(codes), _p(scales), _p(s2), FMT[fmt], LAYOUT[layout],
                                   n_tensors, rows, cols, tensors_per_scale, _p(sum_sq_err), _p(sum_sq_ref),
                                   _p(relerr), _p(workspace), _nbytes(workspace), _stream(stream))
    _check("mxq_dequant_relerr", rc)


def mxq_dequant_relerr_noalloc(x, codes, scales, s2, fmt, n_tensors, rows, cols,
                               tensors_per_scale, sum_sq_err, sum_sq_ref, relerr, stream=None):
    """The verifier without a workspace, for callers that cannot allocate
    device memory: its partial sums live in a fixed 2 MiB array inside the
    library (at most 131072 chunks of 16384 elements per call).  Calls whose
    GPU work overlaps in time share that array and race."""
    _need_verify(x, codes, scales, s2, fmt, "linear", n_tensors, rows, cols, tensors_per_scale,
                 sum_sq_err, sum_sq_ref, relerr)
    rc = load().mxq_dequant_relerr_noalloc(_p(x), _p(codes), _p(scales), _p(s2), FMT[fmt],
                                           n_tensors, rows, cols, tensors_per_scale,
                                           _p(sum_sq_err), _p(sum_sq_ref), _p(relerr),
                                           _stream(stream))
    _check("mxq_dequant_relerr_noalloc", rc)


# The layer operators are called once per layer and token, so their checks are
# kept light.  They run on the device of their first buffer that is not None
# (data of zero bytes may be), whichever device is current, and refuse buffers
# that lie on different ones.
def _first(*bufs):
    for t in bufs:
        if t is not None:
            return t
    raise ValueError("no buffer given")


def _device(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("libmxq takes device tensors")
    return dev


def _buf(name, t, nbytes, dev):
    if t is None:
        return None
    if t.nbytes < nbytes or not t.is_contiguous():
        _need(name, t, nbytes)
    if t.get_device() != dev:
        raise ValueError("%s is not on the device of the first tensor" % name)
    return t.data_ptr()


def _enqueue(fn, args, dev, stream):
    """fn(*args, stream) on device `dev`; stream: a torch stream of it, or its current one."""
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        return fn(*args, raw)
    with torch.cuda.device(dev):
        return fn(*args, raw)


def mxq_quantize_fp8(x, rows, cols, brows, bcols, codes, scales, status, stream=None):
    dev, n = _device(_first(x, status)), rows * cols
    nblk = -(-rows // brows) * -(-cols // bcols) if brows > 0 and bcols > 0 else 0
    rc = _enqueue(load().mxq_quantize_fp8,
                  (_buf("x", x, 2 * n, dev), rows, cols, brows, bcols, _buf("codes", codes, n, dev),
                   _buf("scales", scales, 4 * nblk, dev), _buf("status", status, 4, dev)), dev, stream)
    _check("mxq_quantize_fp8", rc)


def mxq_gemm_fp8(a, a_scales, b, b_scales, M, N, K, out, c, status, stream=None):
    dev, kb = _device(_first(a, status)), -(-K // 128)
    rc = _enqueue(load().mxq_gemm_fp8,
                  (_buf("a", a, M * K, dev), _buf("a_scales", a_scales, 4 * M * kb, dev), _buf("b", b, N * K, dev),
                   _buf("b_scales", b_scales, 4 * -(-N // 128) * kb, dev), M, N, K, OUT[out],
                   _buf("c", c, M * N * (4 if out == "f32" else 2), dev), _buf("status", status, 4, dev)),
                  dev, stream)
    _check("mxq_gemm_fp8", rc)


def moe_weight_bytes(fmt, experts, rows, cols):
    """(codes, scales) bytes of a stack [experts, rows, cols] as mxq_moe_forward reads it."""
    n = experts * rows * cols
    if fmt == "fp8_block":
        return n, 4 * experts * -(-rows // 128) * -(-cols // 128)
    return _code_bytes(fmt, n), n // (16 if fmt == "nvfp4" else 32)


def mxq_moe_forward(x, T, hidden, topk_ids, topk_weights, topk, fmt, experts, inter, gate_up_codes,
                    gate_up_scales, gate_up_s2, down_codes, down_scales, down_s2, y, status, workspace,
                    stream=None):
    dev = _device(_first(x, status))
    gc, gs = moe_weight_bytes(fmt, experts, 2 * inter, hidden)
    dc, ds = moe_weight_bytes(fmt, experts, hidden, inter)
    s2 = 4 * experts if fmt == "nvfp4" else 0
    rc = _enqueue(load().mxq_moe_forward,
                  (_buf("x", x, 2 * T * hidden, dev), T, hidden, _buf("topk_ids", topk_ids, 4 * T * topk, dev),
                   _buf("topk_weights", topk_weights, 4 * T * topk, dev), topk, FMT[fmt], experts, inter,
                   _buf("gate_up_codes", gate_up_codes, gc, dev), _buf("gate_up_scales", gate_up_scales, gs, dev),
                   _buf("gate_up_s2", gate_up_s2, s2, dev), _buf("down_codes", down_codes, dc, dev),
                   _buf("down_scales", down_scales, ds, dev), _buf("down_s2", down_s2, s2, dev),
                   _buf("y", y, 2 * T * hidden, dev), _buf("status", status, 4, dev),
                   _buf("workspace", workspace, 0, dev), _nbytes(workspace)), dev, stream)
    _check("mxq_moe_forward", rc)


def mxq_linear(x, T, K, fmt, codes, scales, s2, N, out, y, status, workspace, stream=None):
    dev = _device(_first(x, status) if x is None else x)
    nb = N * K // (16 if fmt == "nvfp4" else 32)
    rc = _enqueue(load().mxq_linear,
                  (_buf("x", x, 2 * T * K, dev), T, K, FMT[fmt], _buf("codes", codes, _code_bytes(fmt, N * K), dev),
                   _buf("scales", scales, nb, dev), _buf("s2", s2, 4 if fmt == "nvfp4" else 0, dev), N, OUT[out],
                   _buf("y", y, T * N * (4 if out == "f32" else 2), dev), _buf("status", status, 4, dev),
                   _buf("workspace", workspace, 0, dev), _nbytes(workspace)), dev, stream)
    _check("mxq_linear", rc)


class Cache:
    """A paged, quantized key/value cache: the tensors of struct mxq_cache and the
    struct itself.  k_codes, v_codes: uint8 [pages, kv_heads, page_tokens, head_dim]
    ("mxfp8") or [..., head_dim / 2] ("nvfp4"); k_scales, v_scales: uint8 [...,
    head_dim / 32] or [..., head_dim / 16]; k_s2, v_s2: fp32 [kv_heads], the heads'
    global scales ("nvfp4" only).  Contiguous, on one device."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, fmt="mxfp8", k_s2=None, v_s2=None):
        if fmt not in ("mxfp8", "nvfp4"):
            raise ValueError("a cache is mxfp8 or nvfp4, not %r" % (fmt,))
        if k_codes.dim() != 4:
            raise ValueError("codes [pages, kv_heads, page_tokens, ...]")
        pages, heads, tokens, width = k_codes.shape
        dim, block = (width, 32) if fmt == "mxfp8" else (2 * width, 16)
        if dim not in (64, 128, 256) or tokens not in (16, 32, 64, 128, 256):
            raise ValueError("heads of 64, 128 or 256 values on pages of 16, 32, 64, 128 or 256 tokens, not of %d on %d"
                             % (dim, tokens))
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            _typed(name, t, torch.uint8, (pages, heads, tokens, width))
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _typed(name, t, torch.uint8, (pages, heads, tokens, dim // block))
        if fmt == "nvfp4":
            for name, t in (("k_s2", k_s2), ("v_s2", v_s2)):
                _typed(name, t, torch.float32, (heads,))
        else:
            k_s2 = v_s2 = None
        self.tensors = (k_codes, k_scales, v_codes, v_scales, k_s2, v_s2)
        self.device = k_codes.device
        if any(t is not None and t.device != self.device for t in self.tensors):
            raise ValueError("the cache's tensors lie on different devices")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.k_s2, self.v_s2 = self.tensors
        self.fmt, self.pages, self.kv_heads, self.page_tokens, self.head_dim = fmt, pages, heads, tokens, dim
        self.struct = _CacheStruct(*[None if t is None else t.data_ptr() for t in self.tensors], pages, heads, tokens,
                                   dim, FMT[fmt])
        self._ref, self._index = ctypes.byref(self.struct), k_codes.get_device()

    @classmethod
    def empty(cls, pages, kv_heads, page_tokens, head_dim, fmt="mxfp8", k_s2=None, v_s2=None, device="cuda"):
        """A cache of zeros."""
        width, block = (head_dim, 32) if fmt == "mxfp8" else (head_dim // 2, 16)
        make = lambda w: torch.zeros((pages, kv_heads, page_tokens, w), dtype=torch.uint8, device=device)  # noqa: E731
        return cls(make(width), make(head_dim // block), make(width), make(head_dim // block), fmt, k_s2, v_s2)


def _batch(cu, lens, table, seqs, width, dev):
    return (_buf("cu", cu, 4 * (seqs + 1), dev), _buf("lens", lens, 4 * seqs, dev),
            _buf("table", table, 4 * seqs * width, dev), seqs, width)


def _cache_device(cache):
    if cache._index < 0:
        raise ValueError("libmxq takes device tensors")
    return cache._index


def _rows(name, t, stride, T, values, dev):
    """Address of T bf16 rows of `values` contiguous values, `stride` values apart: a contiguous
    buffer, or one whose first dimension is the rows."""
    if t is None:
        return None
    if t.dtype != torch.bfloat16:
        raise ValueError("%s holds %s, not bf16" % (name, t.dtype))
    if T > 0 and t.untyped_storage().nbytes() < (t.storage_offset() + (T - 1) * stride + values) * 2:
        raise ValueError("%s does not hold %d rows of %d values, %d apart" % (name, T, values, stride))
    if T > 0 and not t.is_contiguous():
        shape, strides = t.shape, t.stride()
        n, ok = 1, strides[0] == stride
        for d in range(len(shape) - 1, 0, -1):
            ok &= strides[d] == n or shape[d] == 1
            n *= shape[d]
        if not ok or n != values:
            raise ValueError("the rows of %s are not of %d contiguous values, %d apart" % (name, values, stride))
    if t.get_device() != dev:
        raise ValueError("%s is not on the device of the first tensor" % name)
    return t.data_ptr()


def mxq_cache_write(cache, k, k_stride, v, v_stride, T, cu, lens, table, seqs, width, mode, status, stream=None):
    """k and v: bf16 tensors whose row t starts t * stride values behind their first
    value and holds kv_heads * head_dim contiguous ones."""
    dev, n = _cache_device(cache), cache.kv_heads * cache.head_dim
    rc = _enqueue(load().mxq_cache_write,
                  (cache._ref, _rows("k", k, k_stride, T, n, dev), k_stride, _rows("v", v, v_stride, T, n, dev), v_stride,
                   T, *_batch(cu, lens, table, seqs, width, dev), SCALE_MODE[mode], _buf("status", status, 4, dev)),
                  dev, stream)
    _check("mxq_cache_write", rc)


def mxq_cache_read(cache, cu, lens, table, seqs, width, T, k, v, status, stream=None):
    dev, n = _cache_device(cache), 2 * T * cache.kv_heads * cache.head_dim
    rc = _enqueue(load().mxq_cache_read,
                  (cache._ref, *_batch(cu, lens, table, seqs, width, dev), T, _buf("k", k, n, dev),
                   _buf("v", v, n, dev), _buf("status", status, 4, dev)), dev, stream)
    _check("mxq_cache_read", rc)


def mxq_cache_attention(cache, q, q_stride, T, heads, cu, lens, table, seqs, width, max_new, scale, o, lse, status,
                        workspace, stream=None):
    """q: bf16, row t `t * q_stride` values behind the first, heads * head_dim contiguous ones each."""
    dev, n = _cache_device(cache), heads * cache.head_dim
    rc = _enqueue(load().mxq_cache_attention,
                  (cache._ref, _rows("q", q, q_stride, T, n, dev), q_stride, T, heads,
                   *_batch(cu, lens, table, seqs, width, dev), max_new, scale, _buf("o", o, 2 * T * n, dev),
                   _buf("lse", lse, 4 * T * heads, dev), _buf("status", status, 4, dev),
                   _buf("workspace", workspace, 0, dev), _nbytes(workspace)), dev, stream)
    _check("mxq_cache_attention", rc)


# ------------------------------------------------------------ allocating --
def _on(stream):
    """Results and workspaces made on the stream that the call runs on: what is
    freed on return is then handed out again only behind the call."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _bf16(x):
    if x.dtype != torch.bfloat16 or not x.is_contiguous():
        raise ValueError("expected a contiguous bf16 tensor")
    return x


def quantize_nvfp4(x, mode="four_six", with_mbits=True, stream=None, layout="linear"):
    """x: bf16 [G, R, C] on the device.  Returns a dict of device tensors:
    codes [G,R,C/2] u8, scales ([G,R,C/16] u8 when linear, the flat tiled
    bytes of G matrices when layout="swizzled_128x4"), s2 [G] f32, mbits u32
    words, m4_count [G] i32-view of u32, status [1]."""
    _bf16(x)
    G, R, C = x.shape
    dev = x.device
    out = {
        "codes": torch.empty((G, R, C // 2), dtype=torch.uint8, device=dev),
        "scales": torch.empty((G, R, C // 16), dtype=torch.uint8, device=dev) if layout == "linear"
        else torch.empty(max(scale_bytes("nvfp4", layout, G, R, C), 1), dtype=torch.uint8, device=dev),
        "s2": torch.empty(G, dtype=torch.float32, device=dev),
        "mbits": torch.empty(((G * R * C // 16) + 31) // 32 or 1, dtype=torch.int32, device=dev)
        if with_mbits else None,
        "m4_count": torch.empty(max(G, 1), dtype=torch.int32, device=dev),
        "status": torch.zeros(1, dtype=torch.int32, device=dev),
    }
    ws, _ = _workspace("quantize_nvfp4", G, R, C, dev)
    mxq_quantize_nvfp4(x, G, R, C, mode, layout, out["codes"], out["scales"], out["s2"],
                       out["mbits"], out["m4_count"], out["status"], ws, stream)
    return out


def quantize_nvfp4_s2(x, s2_in, mode="four_six", with_mbits=True, stream=None, layout="linear"):
    """x: bf16 [G, R, C]; s2_in: fp32 [G] global scales on the device (gate
    and up held apart pass the scale they share).  Returns a dict of device
    tensors: codes, scales, mbits, m4_count, status (as quantize_nvfp4,
    without s2)."""
    _bf16(x)
    G, R, C = x.shape
    if s2_in.dtype != torch.float32 or not s2_in.is_contiguous() or s2_in.numel() < G:
        raise ValueError("expected contiguous fp32 global scales [G]")
    dev = x.device
    out = {
        "codes": torch.empty((G, R, C // 2), dtype=torch.uint8, device=dev),
        "scales": torch.empty((G, R, C // 16), dtype=torch.uint8, device=dev) if layout == "linear"
        else torch.empty(max(scale_bytes("nvfp4", layout, G, R, C), 1), dtype=torch.uint8, device=dev),
        "mbits": torch.empty(((G * R * C // 16) + 31) // 32 or 1, dtype=torch.int32, device=dev)
        if with_mbits else None,
        "m4_count": torch.empty(max(G, 1), dtype=torch.int32, device=dev),
        "status": torch.zeros(1, dtype=torch.int32, device=dev),
    }
    mxq_quantize_nvfp4_s2(x, G, R, C, s2_in, mode, layout, out["codes"], out["scales"], out["mbits"],
                          out["m4_count"], out["status"], stream)
    return out


def global_scale_nvfp4(x, stream=None):
    """x: bf16 [G, R, C].  Returns (s2 [G] fp32, status [1]) on the device:
    s2 = RN32(amax_g / 2688) per group."""
    _bf16(x)
    G, R, C = x.shape
    s2 = torch.empty(max(G, 1), dtype=torch.float32, device=x.device)
    status = torch.zeros(1, dtype=torch.int32, device=x.device)
    mxq_global_scale_nvfp4(x, G, R, C, s2, status, stream)
    return s2[:G], status


class Census:
    """A device-resident struct mxq_census: reset on creation, filled by
    add() (mxq_census_add), read by result() (one small device -> host
    copy, after which the struct's fields come back as a dict)."""

    def __init__(self, device="cuda", stream=None):
        self.buf = torch.empty(len(CENSUS_FIELDS), dtype=torch.float64, device=device)
        mxq_census_reset(self.buf, stream)

    def add(self, n_tensors=0, sum_sq_err=None, sum_sq_ref=None, relerr=None, sum_sq_err_rtn=None,
            n_groups=0, m4_count=None, blocks_per_group=0, stream=None):
        mxq_census_add(self.buf, n_tensors, sum_sq_err, sum_sq_ref, relerr, sum_sq_err_rtn, n_groups,
                       m4_count, blocks_per_group, stream)

    def result(self):
        raw = self.buf.cpu()
        ints = raw.view(torch.int64)
        return {k: (int(ints[i]) if k in _CENSUS_INTS else float(raw[i]))
                for i, k in enumerate(CENSUS_FIELDS) if k != "reserved"}


def quantize_nvfp4_weighted(x, h, stream=None, layout="linear"):
    """x: bf16 [G, R, C]; h: fp32 weights per input channel, [C] (shared) or
    [G, C].  Returns dict codes, scales, s2, status."""
    _bf16(x)
    G, R, C = x.shape
    if h.dtype != torch.float32 or not h.is_contiguous() or h.shape[-1] != C:
        raise ValueError("expected contiguous fp32 weights [C] or [G, C]")
    hg = 1 if h.dim() == 1 else h.shape[0]
    dev = x.device
    out = {
        "codes": torch.empty((G, R, C // 2), dtype=torch.uint8, device=dev),
        "scales": torch.empty((G, R, C // 16), dtype=torch.uint8, device=dev) if layout == "linear"
        else torch.empty(max(scale_bytes("nvfp4", layout, G, R, C), 1), dtype=torch.uint8, device=dev),
        "s2": torch.empty(max(G, 1), dtype=torch.float32, device=dev),
        "status": torch.zeros(1, dtype=torch.int32, device=dev),
    }
    ws, _ = _workspace("quantize_nvfp4", G, R, C, dev)
    mxq_quantize_nvfp4_weighted(x, G, R, C, h, hg, layout, out["codes"], out["scales"], out["s2"],
                                out["status"], ws, stream)
    return out


def quantize_mx(x, fmt, stream=None, layout="linear"):
    """x: bf16 [..., C], quantized as one [rows, C] matrix.  Returns dict
    codes, scales (tiled bytes of that one matrix when layout is
    "swizzled_128x4"), status."""
    _bf16(x)
    C = x.shape[-1]
    R = x.numel() // C if C else 0
    dev = x.device
    out = {
        "codes": torch.empty(x.shape[:-1] + ((C // 2) if fmt == "mxfp4" else C,), dtype=torch.uint8,
                             device=dev),
        "scales": torch.empty(x.shape[:-1] + (C // 32,), dtype=torch.uint8, device=dev)
        if layout == "linear"
        else torch.empty(max(scale_bytes(fmt, layout, 1, R, C), 1), dtype=torch.uint8, device=dev),
        "status": torch.zeros(1, dtype=torch.int32, device=dev),
    }
    mxq_quantize_mx(x, R, C, fmt, 32, layout, out["codes"], out["scales"], out["status"], stream)
    return out


def requant_fp8_mx(fp8, bscale, brows, bcols, fmt, stream=None, layout="linear"):
    """fp8: uint8 E4M3 codes [R, C] on the device; bscale: fp32
    [ceil(R/brows), ceil(C/bcols)].  Returns dict codes, scales, status."""
    if fp8.dtype != torch.uint8 or not fp8.is_contiguous() or fp8.dim() != 2:
        raise ValueError("expected a contiguous uint8 [rows, cols] tensor of E4M3 codes")
    if bscale.dtype != torch.float32 or not bscale.is_contiguous():
        raise ValueError("expected contiguous fp32 block scales")
    R, C = fp8.shape
    dev = fp8.device
    out = {
        "codes": torch.empty((R, (C // 2) if fmt == "mxfp4" else C), dtype=torch.uint8, device=dev),
        "scales": torch.empty((R, C // 32), dtype=torch.uint8, device=dev) if layout == "linear"
        else torch.empty(max(scale_bytes(fmt, layout, 1, R, C), 1), dtype=torch.uint8, device=dev),
        "status": torch.zeros(1, dtype=torch.int32, device=dev),
    }
    mxq_requant_fp8_mx(fp8, bscale, R, C, brows, bcols, fmt, layout, out["codes"], out["scales"],
                       out["status"], stream)
    return out


def quantize_fp8(x, brows=1, stream=None):
    """x: bf16 [..., C], quantized as one [rows, C] matrix to E4M3 with one
    fp32 scale per brows x 128 block (1: token tiles, 128: weights).  Returns
    dict codes [..., C] u8, scales [ceil(rows/brows), ceil(C/128)] f32 (a stack
    [E, R, C] of weights with R a multiple of 128: [E, R/128, ceil(C/128)]),
    status."""
    _bf16(x)
    if brows not in (1, 128):
        raise ValueError("blocks of 1 x 128 or 128 x 128")
    C = x.shape[-1]
    R = x.shape[:-1].numel()
    lead = (-(-R // brows),)
    if x.dim() == 3 and brows == 128 and x.shape[1] % 128 == 0:
        lead = (x.shape[0], x.shape[1] // 128)
    dev = x.device
    with _on(stream):
        out = {
            "codes": torch.empty(x.shape, dtype=torch.uint8, device=dev),
            "scales": torch.empty(lead + (-(-C // 128),), dtype=torch.float32, device=dev),
            "status": torch.zeros(1, dtype=torch.int32, device=dev),
        }
        mxq_quantize_fp8(x, R, C, brows, 128, out["codes"], out["scales"], out["status"], stream)
    return out


def gemm_fp8(a, a_scales, b, b_scales, out="bf16", status=None, stream=None):
    """c = a b^T of block-FP8 matrices.  a: uint8 E4M3 codes [M, K] with fp32
    scales [M, ceil(K/128)] (quantize_fp8 of a token tile); b: codes [N, K]
    with scales [ceil(N/128), ceil(K/128)] (brows=128).  Returns dict c [M, N]
    (bf16, or fp32 for out="f32"), status (a given one is added to)."""
    M, K = a.shape
    N = b.shape[0]
    kb = -(-K // 128)
    _typed("a", a, torch.uint8, (M, K))
    _typed("a_scales", a_scales, torch.float32, (M, kb))
    _typed("b", b, torch.uint8, (N, K))
    _typed("b_scales", b_scales, torch.float32, (-(-N // 128), kb))
    if out not in OUT:
        raise ValueError("out is one of %s" % sorted(OUT))
    with _on(stream):
        res = {"c": torch.empty((M, N), dtype=torch.float32 if out == "f32" else torch.bfloat16, device=a.device),
               "status": torch.zeros(1, dtype=torch.int32, device=a.device) if status is None else status}
        mxq_gemm_fp8(a, a_scales, b, b_scales, M, N, K, out, res["c"], res["status"], stream)
    return res


def moe_workspace(T, topk, hidden, inter, device="cuda"):
    """A workspace for mxq_moe_forward at these sizes, to keep from call to call."""
    return torch.empty(max(load().mxq_moe_workspace_bytes(T, topk, hidden, inter), 256), dtype=torch.uint8,
                       device=device)


def _typed(name, t, dtype, shape):
    if t is None or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("expected %s as contiguous %s %s" % (name, dtype, list(shape)))
    return t


def moe_forward(x, topk_ids, topk_weights, gate_up, down, fmt, workspace=None, stream=None):
    """A routed-expert layer for a few tokens.  x: bf16 [T, H]; topk_ids int32
    and topk_weights fp32 [T, k] (an id below 0: no expert); gate_up, down:
    dicts with codes, scales (and s2 for "nvfp4") of the stacks [E, 2I, H] and
    [E, H, I], as quantize_nvfp4, quantize_mx or quantize_fp8 with brows=128
    (fmt "fp8_block") return them with linear scales; workspace: a
    moe_workspace to use again, not by two calls at once.  Returns dict y bf16
    [T, H], status."""
    _bf16(x)
    per = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32, "fp8_block": 128}.get(fmt)
    if per is None:
        raise ValueError("unknown format %r" % (fmt,))
    T, H = x.shape
    E, I = gate_up["codes"].shape[0], gate_up["codes"].shape[1] // 2
    k = topk_ids.shape[1]
    _typed("topk_ids", topk_ids, torch.int32, (T, k))
    _typed("topk_weights", topk_weights, torch.float32, (T, k))
    for name, q, rows, cols in (("gate_up", gate_up, 2 * I, H), ("down", down, H, I)):
        _typed(name + " codes", q["codes"], torch.uint8,
               (E, rows, cols // 2 if fmt in ("nvfp4", "mxfp4") else cols))
        if fmt == "fp8_block":
            _typed(name + " scales", q["scales"], torch.float32, (E, -(-rows // per), -(-cols // per)))
        else:
            _typed(name + " scales", q["scales"], torch.uint8, (E, rows, cols // per))
        if fmt == "nvfp4":
            _typed(name + " s2", q["s2"], torch.float32, (E,))
    dev = x.device
    with _on(stream):
        out = {"y": torch.empty((T, H), dtype=torch.bfloat16, device=dev),
               "status": torch.zeros(1, dtype=torch.int32, device=dev)}
        mxq_moe_forward(x, T, H, topk_ids, topk_weights, k, fmt, E, I, gate_up["codes"], gate_up["scales"],
                        gate_up["s2"] if fmt == "nvfp4" else None, down["codes"], down["scales"],
                        down["s2"] if fmt == "nvfp4" else None, out["y"], out["status"],
                        moe_workspace(T, k, H, I, dev) if workspace is None else workspace, stream)
    return out


def linear_workspace(T, K, device="cuda"):
    """A workspace for mxq_linear at these sizes, to keep from call to call."""
    return torch.empty(max(load().mxq_linear_workspace_bytes(T, K), 256), dtype=torch.uint8, device=device)


LINEAR_MAX_TOKENS = 2048        # of one call of mxq_linear


def linear(x, w, fmt, out="bf16", workspace=None, stream=None, y=None, status=None):
    """x w^T for a few tokens over a quantized matrix.  x: bf16 [T, K]; w: a dict with
    codes, scales (and s2 [1] for "nvfp4") of the matrix [N, K] as quantize_nvfp4 (of
    [1, N, K]) or quantize_mx return it with linear scales; workspace: a
    linear_workspace to use again, not by two calls at once; y: the result's tensor, where
    the caller has one.  Returns dict y [T, N] (bf16, or fp32 for out="f32"), status (a
    given one is added to)."""
    _bf16(x)
    per = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}.get(fmt)
    if per is None:
        raise ValueError("unknown format %r" % (fmt,))
    if out not in OUT:
        raise ValueError("out is one of %s" % sorted(OUT))
    T, K = x.shape
    codes = w["codes"][0] if w["codes"].dim() == 3 and w["codes"].shape[0] == 1 else w["codes"]
    scales = w["scales"][0] if w["scales"].dim() == 3 and w["scales"].shape[0] == 1 else w["scales"]
    N = codes.shape[0]
    _typed("codes", codes, torch.uint8, (N, K if fmt == "mxfp8" else K // 2))
    _typed("scales", scales, torch.uint8, (N, K // per))
    if fmt == "nvfp4":
        _typed("s2", w["s2"], torch.float32, (1,))
    dev, dtype = x.device, torch.float32 if out == "f32" else torch.bfloat16
    if y is not None:
        _typed("y", y, dtype, (T, N))
    with _on(stream):
        res = {"y": torch.empty((T, N), dtype=dtype, device=dev) if y is None else y,
               "status": torch.zeros(1, dtype=torch.int32, device=dev) if status is None else status}
        mxq_linear(x, T, K, fmt, codes, scales, w["s2"] if fmt == "nvfp4" else None, N, out, res["y"], res["status"],
                   linear_workspace(T, K, dev) if workspace is None else workspace, stream)
    return res


def _token_rows(name, t, heads, dim):
    """(rows, stride) of a bf16 [T, heads, dim] tensor whose tokens may lie apart."""
    if t.dtype != torch.bfloat16 or t.dim() != 3 or tuple(t.shape[1:]) != (heads, dim):
        raise ValueError("expected %s as bf16 [T, %d, %d]" % (name, heads, dim))
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim):
        raise ValueError("a token's heads must be contiguous in %s" % name)
    return t.shape[0], (t.stride(0) if t.shape[0] > 1 else heads * dim)


def _batch_of(cu, lens, table):
    """(sequences, width of the table) of a batch."""
    B = lens.shape[0] if lens.dim() == 1 else -1
    _typed("cu", cu, torch.int32, (B + 1,))
    _typed("lens", lens, torch.int32, (B,))
    if table.dim() != 2:
        raise ValueError("table is [sequences, pages of the longest]")
    _typed("table", table, torch.int32, (B, table.shape[1]))
    return B, table.shape[1]


def cache_write(cache, k, v, cu, lens, table, mode="rtn", status=None, stream=None):
    """Quantize the keys and values of the batch's new tokens into the cache.  k, v:
    bf16 [T, kv_heads, head_dim], a token's heads contiguous; cu int32 [B + 1], lens
    int32 [B], table int32 [B, width]: see include/mxq.h.  mode: block scales of
    "nvfp4", "rtn" or "four_six".  Returns the status (a given one is added to)."""
    T, ks = _token_rows("k", k, cache.kv_heads, cache.head_dim)
    Tv, vs = _token_rows("v", v, cache.kv_heads, cache.head_dim)
    if T != Tv:
        raise ValueError("%d keys and %d values" % (T, Tv))
    B, width = _batch_of(cu, lens, table)
    with _on(stream):
        status = torch.zeros(1, dtype=torch.int32, device=cache.device) if status is None else status
        mxq_cache_write(cache, k, ks, v, vs, T, cu, lens, table, B, width, mode, status, stream)
    return status


def cache_read(cache, cu, lens, table, T, stream=None):
    """The last tokens of the batch's sequences back from the cache: dict k, v bf16
    [T, kv_heads, head_dim] (rows of no sequence, or without a place, are zeros),
    status.  With cu the running sum of lens: whole sequences."""
    B, width = _batch_of(cu, lens, table)
    with _on(stream):
        out = {n: torch.zeros((T, cache.kv_heads, cache.head_dim), dtype=torch.bfloat16, device=cache.device) for n in "kv"}
        out["status"] = torch.zeros(1, dtype=torch.int32, device=cache.device)
        mxq_cache_read(cache, cu, lens, table, B, width, T, out["k"], out["v"], out["status"], stream)
    return out


def cache_attention_workspace(cache, T, heads, seqs, max_new):
    """A workspace for mxq_cache_attention at these sizes, to keep from call to call."""
    n = load().mxq_cache_attention_workspace_bytes(cache.struct, T, heads, seqs, max_new)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=cache.device)


def cache_attention(cache, q, cu, lens, table, max_new, scale=None, workspace=None, status=None, stream=None):
    """Causal attention of the batch's new tokens over the cache, which holds their
    own keys and values already.  q: bf16 [T, heads, head_dim], a token's heads
    contiguous; max_new: no sequence has more new tokens; scale: 1 / sqrt(head_dim)
    where None; workspace: a cache_attention_workspace to use again, not by two calls
    at once.  Returns dict o bf16 [T, heads, head_dim], lse fp32 [T, heads] (rows of
    no sequence: zeros), status (a given one is added to)."""
    if q.dim() != 3:
        raise ValueError("expected q as bf16 [T, heads, head_dim]")
    heads = q.shape[1]
    T, qs = _token_rows("q", q, heads, cache.head_dim)
    B, width = _batch_of(cu, lens, table)
    dev = cache.device
    with _on(stream):
        out = {"o": torch.zeros((T, heads, cache.head_dim), dtype=torch.bfloat16, device=dev),
               "lse": torch.zeros((T, heads), dtype=torch.float32, device=dev),
               "status": torch.zeros(1, dtype=torch.int32, device=dev) if status is None else status}
        if workspace is None:
            workspace = cache_attention_workspace(cache, T, heads, B, max_new)
        mxq_cache_attention(cache, q, qs, T, heads, cu, lens, table, B, width, max_new,
                            cache.head_dim ** -0.5 if scale is None else scale, out["o"], out["lse"], out["status"],
                            workspace, stream)
    return out


def quantize_act(tokens, fmt, stream=None, mode="rtn", layout="linear"):
    """tokens: bf16 [T, hidden].  NVFP4 returns input_scale too; mode
    "four_six" applies the 4/6-optimal block scales to the tile."""
    _bf16(tokens)
    T, H = tokens.shape
    dev = tokens.device
    blk = 16 if fmt == "nvfp4" else 32
    out = {
        "codes": torch.empty((T, H if fmt == "mxfp8" else H // 2), dtype=torch.uint8, device=dev),
        "scales": torch.empty((T, H // blk), dtype=torch.uint8, device=dev) if layout == "linear"
        else torch.empty(max(scale_bytes(fmt, layout, 1, T, H), 1), dtype=torch.uint8, device=dev),
        "input_scale": torch.empty(1, dtype=torch.float32, device=dev),
        "status": torch.zeros(1, dtype=torch.int32, device=dev),
    }
    ws, _ = _workspace("quantize_act", T, H, 0, dev)
    mxq_quantize_act(tokens, T, H, fmt, mode, layout, out["codes"], out["scales"],
                     out["input_scale"], out["status"], ws, stream)
    return out


def dequant_relerr(x, codes, scales, s2, fmt, n_tensors, rows, cols, tensors_per_scale=1,
                   stream=None, layout="linear"):
    """Per-tensor fp64 (sum_sq_err, sum_sq_ref, relerr) on the device."""
    dev = x.device
    err = torch.empty(max(n_tensors, 1), dtype=torch.float64, device=dev)
    ref = torch.empty_like(err)
    rel = torch.empty_like(err)
    ws, _ = _workspace("dequant_relerr", n_tensors, rows, cols, dev)
    mxq_dequant_relerr(x, codes, scales, s2, fmt, layout, n_tensors, rows, cols, tensors_per_scale,
                       err, ref, rel, ws, stream)
    return err[:n_tensors], ref[:n_tensors], rel[:n_tensors]

"""What the layer operators refuse or take on the host, without a GPU (the compute entry points are replaced by the
recorder of test_layer_ops_host; host tensors stand in for device tensors)."""
import pytest
import torch

from mxfp_block_scaled_b200 import layers, mxq
from test_layer_ops_host import bf16, lib, rec, tokens, u8      # noqa: F401 -- fixtures


@pytest.mark.parametrize("I", [128, 256, 384])
def test_a_block_fp8_layer_can_be_run(rec, I):      # noqa: F811
    q = layers.block_fp8_layer(bf16(3, 2 * I, 256), bf16(3, 256, I))
    layers.routed_forward(q, *tokens())
    assert [c[0] for c in rec.calls][-1] == "mxq_moe_forward"


@pytest.mark.parametrize("H,I", [(256, 192), (256, 64), (192, 128), (256, 320)])
def test_block_fp8_layers_that_could_not_be_run_are_refused(rec, H, I):     # noqa: F811
    """Blocks that straddle gate and up, or rows of the down slab that end inside a block."""
    with pytest.raises(ValueError, match="multiples of 128"):
        layers.block_fp8_layer(bf16(3, 2 * I, H), bf16(3, H, I))
    assert not rec.calls


def test_slabs_of_different_layers_are_refused(rec):        # noqa: F811
    for gu, dn in (((3, 256, 256), (2, 256, 128)), ((3, 256, 256), (3, 128, 128)), ((3, 256, 256), (3, 256, 256))):
        with pytest.raises(ValueError):
            layers.block_fp8_layer(bf16(*gu), bf16(*dn))
    with pytest.raises(ValueError, match="stack"):
        layers.block_fp8_layer(torch.zeros((256, 256), dtype=torch.bfloat16), bf16(3, 256, 128))
    assert not rec.calls


def test_data_of_zero_bytes_may_be_none(rec):        # noqa: F811
    st = torch.zeros(1, dtype=torch.int32)
    mxq.mxq_quantize_fp8(None, 0, 128, 1, 128, None, None, st)
    mxq.mxq_gemm_fp8(None, None, None, None, 3, 5, 0, "f32", torch.zeros(15), st)
    mxq.mxq_gemm_fp8(None, None, u8(5, 128), torch.zeros(1, 1), 0, 5, 128, "f32", None, st)
    mxq.mxq_moe_forward(None, 0, 256, None, None, 2, "mxfp8", 3, 128, None, None, None, None, None, None, None, st, None)
    assert [c[1][0] for c in rec.calls] == [None] * 4


def test_missing_buffers_get_the_librarys_status(monkeypatch, lib):     # noqa: F811
    """Not an error of the binding: the library refuses them before it enqueues anything."""
    monkeypatch.setattr(mxq, "_device", lambda t: t.get_device())
    monkeypatch.setattr(mxq, "_enqueue", lambda fn, args, dev, stream: fn(*args, None))
    st = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: mxq.mxq_quantize_fp8(None, 4, 128, 1, 128, u8(4, 128), torch.zeros(4), st),
                 lambda: mxq.mxq_gemm_fp8(None, torch.zeros(4), u8(8, 128), torch.zeros(1), 4, 8, 128, "f32", torch.zeros(32), st),
                 lambda: mxq.mxq_moe_forward(None, 2, 256, torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2)), 2, "mxfp8",
                                             3, 128, u8(3, 256, 256), u8(3, 256, 8), None, u8(3, 256, 128), u8(3, 256, 4), None,
                                             bf16(2, 256), st, None)):
        with pytest.raises(mxq.MxqError, match="invalid argument"):
            call()
    with pytest.raises(ValueError, match="no buffer"):
        mxq.mxq_quantize_fp8(None, 4, 128, 1, 128, None, None, None)

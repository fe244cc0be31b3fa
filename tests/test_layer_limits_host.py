"""What the layer operators refuse or take on the host, without a GPU (the compute entry points are replaced by the
recorder of test_layer_ops_host; host tensors stand in for device tensors)."""
import pytest
import torch

from mxfp_block_scaled_b200 import layers
from test_layer_ops_host import bf16, lib, rec, tokens      # noqa: F401 -- fixtures


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

"""Each layer call refuses the expert formats that it does not compute, by name and before anything else."""
import pytest
import torch

import bit_quantized_moe_token_b200 as moe

W = [None] * 6
W4, F8, F4, MX = (moe.Layer(8, 256, 128, *W), moe.Layer8(8, 256, 128, *W), moe.Layer4(8, 256, 128, *W, *W[:3]),
                  moe.LayerMX(8, 256, 128, *W))
HYBRID = moe.LayerH(8, F4, W4, None, None)


def test_forward():
    for call in (lambda: moe.forward(MX, None, None, 2), lambda: moe.forward(MX, None, None, 2, out=0, ws=0),
                 lambda: moe.alloc_workspace(MX, 4, 2, "cpu")):
        with pytest.raises(ValueError, match="forward: expected a layer of type Layer or Layer8 or Layer4 or LayerH"):
            call()


@pytest.mark.parametrize("layer", [F8, F4, HYBRID, None])
def test_few_token_layer(layer):
    for call in (lambda: moe.decode(layer, None, None, 2), lambda: moe.decode(layer, None, None, 2, out=0, ws=0),
                 lambda: moe.decode_router(layer, None, None, 2, out=0, ws=0),
                 lambda: moe.alloc_decode_workspace(layer, 4, 2, "cpu")):
        with pytest.raises(ValueError, match="decode(_router)?: expected a layer of type Layer or LayerMX"):
            call()


@pytest.mark.parametrize("fmt,layer", [("w4a8", MX), ("w4a8", F8), ("mxfp4", W4), ("mxfp4", F4)])
def test_entry_points(fmt, layer):
    for tail in ("decode", "decode_router"):
        with pytest.raises(ValueError, match=f"moe_{fmt}_decode: expected a"):
            getattr(moe, f"moe_{fmt}_{tail}")(layer, None, None, 2, None, None)


def test_a_program_s_own_kind_of_layer_stays():
    """forward and its workspace take what has a W4A8 layer's attributes, as before."""
    class Own:
        shape_struct = W4.shape_struct
        gate_packed = None

    assert moe.alloc_workspace(Own(), 4, 2, "cpu").numel() == moe.alloc_workspace(W4, 4, 2, "cpu").numel()


def test_the_formats_that_are_computed_get_their_workspace():
    for layer in (W4, F8, F4):
        assert moe.alloc_workspace(layer, 4, 2, "cpu").numel() > 0
    for layer in (W4, MX):
        assert moe.alloc_decode_workspace(layer, 4, 2, "cpu").numel() > 0


def test_product_of_one_type_into_another():
    out = torch.empty(2, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="but out is"):
        moe.matmul_mxfp4(None, None, None, None, dtype=torch.float32, out=out)

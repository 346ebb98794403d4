"""What distill.py refuses before it reaches a GPU (CPU)."""
import pytest

torch = pytest.importorskip("torch")
distill = pytest.importorskip("post_weight_quantization_amd.distill")


def _layer():
    return distill.I8Linear(torch.zeros(3, 128, dtype=torch.int8), torch.ones(3), 8)


def test_the_8_bit_layer_refuses_to_lose_a_gradient():
    x = torch.zeros(4, 8, requires_grad=True)
    with pytest.raises(ValueError, match="^x: expected a tensor that needs no gradient"):
        _layer()(x)
    with pytest.raises(ValueError, match="^x: expected a tensor that needs no gradient"):
        _layer()(2.0 * x)
    # where none is recorded, or asked for, the call goes on (to the check of the device)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        _layer()(x)
    with pytest.raises(ValueError, match="GPU"):
        _layer()(x.detach())

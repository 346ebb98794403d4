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


@pytest.mark.parametrize("which", ["weight", "values", "lse"])
def test_the_loss_refuses_gradients_it_does_not_compute(which):
    t = dict(weight=torch.ones(4), values=torch.zeros(4, 2), lse=torch.zeros(4))
    t[which].requires_grad_()
    teacher = distill.TeacherTop(t["values"], torch.zeros(4, 2, dtype=torch.int32), t["lse"])
    logits = torch.zeros(4, 9, requires_grad=True)
    with pytest.raises(ValueError, match=f"^{which}: expected a tensor that needs no gradient"):
        distill.distill_loss(logits, teacher, t["weight"])
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        distill.distill_loss(logits, teacher, t["weight"])

"""GPU tests of the distillation loss in torch's autograd: what it keeps between
the forward and the backward pass."""
import numpy as np
import pytest

from oracle import head
from tests.gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

if have_gpu():
    import torch

    from post_weight_quantization_amd import distill


@pytest.mark.parametrize("which", ["values", "index", "lse", "weight"])
def test_answers_written_before_the_backward_pass_are_noticed(which):
    """A buffer of answers that the next batch overwrites must not change the
    gradient of this one in silence."""
    torch.manual_seed(0)
    logits = torch.randn(6, 300, device="cuda", requires_grad=True)
    t = distill.teacher_top(torch.randn(6, 300, device="cuda") * 3, 8)
    weight = torch.rand(6, device="cuda")
    loss = distill.distill_loss(logits, t, weight).sum()
    (weight if which == "weight" else getattr(t, which)).add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("rest", [False, True])
def test_two_losses_of_one_logits(rest):
    """Two teachers, two temperatures, one backward pass: the gradients add up."""
    torch.manual_seed(1)
    n, v = 10, 777
    logits = torch.randn(n, v, device="cuda", requires_grad=True)
    want, total = np.zeros((n, v)), 0.0
    for T, k, up in ((1.0, 5, 1.0), (2.0, 40, 0.5)):
        t = distill.teacher_top(torch.randn(n, v, device="cuda") * 3, k, T, rest=rest)
        total = total + up * distill.distill_loss(logits, t).sum()
        _, g, _ = head.distill(host(logits), host(t.values), host(t.index), host(t.lse) if rest else None, T)
        want += up * g
    total.backward()
    # each loss's gradient within w T 1e-4 (q (1 + r / q_r) + p), terms of which add up to 4
    assert np.abs(host(logits.grad) - want).max() <= 2 * 4e-4

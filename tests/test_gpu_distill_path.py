"""The 8-bit layer, the teacher's top logits and the distillation loss used
together (distill.py), against oracle/head.py and the oracle's covariances.

Losses and gradients are held to the bounds of the parity tests of the
entry points; covariances to 1e-4 relative Frobenius, as in the other parity
tests; the sensitivity to 1e-5 of the traces of the same matrices.
"""
import numpy as np
import pytest

import oracle
from oracle import head
from tests.gpu_util import dev, have_gpu, host, rel_fro

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

if have_gpu():
    import torch

    import post_weight_quantization_amd as kq
    from post_weight_quantization_amd import distill


def _np(t):
    return host(t.float()) if t.dtype == torch.bfloat16 else host(t)


def test_sweep_at_8_bits_serves_through_the_8_bit_layer():
    """Covariances, factor, 8-bit sweep without incoherence processing, and the
    8-bit product with its codes."""
    rng = np.random.default_rng(0)
    n, m, d = 512, 96, 256
    x = (rng.standard_normal((n, d)) * np.exp(rng.normal(0, 1, d))).astype(np.float32)
    W = (rng.standard_normal((m, d)) * 0.02).astype(np.float32)
    HX, _, _ = kq.kq_accumulate_cov(None, dev(x), None, 1.0 / n, 0.0, want=("HX",))
    U = kq.kq_cholesky_inv(HX, 0.01)
    Wq = dev(W)
    codes, scale, zero = kq.kq_gptaq_quantize(Wq, U, None, 8)
    layer = distill.I8Linear.from_codes(codes, scale, zero)
    y = layer(dev(x[:40]).reshape(5, 8, d))
    assert y.shape == (5, 8, m)
    c, s, _ = head.quantize_rows(x[:40])
    want, _ = head.product(c, s, host(codes).astype(int), host(scale)[:, 0], host(zero)[:, 0])
    assert np.all(np.abs(host(y).reshape(40, m) - want) <= 4 * 2.0 ** -24 * np.abs(want) + 1e-37)
    # near the layer itself: half a step of each grid over the row
    exact = x[:40].astype(np.float64) @ W.T.astype(np.float64)
    bound = 0.5 * s[:, None] * np.abs(host(Wq)).sum(1)[None, :]
    sweep = np.abs(x[:40].astype(np.float64) @ (host(Wq) - W).T.astype(np.float64))
    assert np.all(np.abs(host(y).reshape(40, m) - exact) <= bound + sweep + 1e-4)


def test_rounded_to_nearest_layer():
    rng = np.random.default_rng(1)
    W = (rng.standard_normal((50, 333)) * 0.1).astype(np.float32)
    b = rng.standard_normal(50).astype(np.float32)
    layer = distill.I8Linear.from_weight(dev(W), dev(b))
    x = rng.standard_normal((7, 333)).astype(np.float32)
    wc, ws, _ = head.quantize_rows(W)
    np.testing.assert_array_equal(host(layer.codes)[:, :333], wc)
    c, s, _ = head.quantize_rows(x)
    want, _ = head.product(c, s, wc, ws, None, b)
    assert np.all(np.abs(host(layer(dev(x))) - want) <= 4 * 2.0 ** -24 * (np.abs(want) + 2 * np.abs(b)) + 1e-37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rest", [False, True])
def test_loss_in_autograd(rest, dtype):
    """A mean over weighted tokens, back through a linear layer."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    torch.manual_seed(2)
    n, d, v, k = (2, 12), 64, 1000, 16
    lin = torch.nn.Linear(d, v).to("cuda", dt)
    x = torch.randn(*n, d, device="cuda").to(dt)
    teacher_logits = torch.randn(*n, v, device="cuda") * 3
    t = distill.teacher_top(teacher_logits, k, 2.0, rest=rest)
    w = torch.rand(*n, device="cuda")
    w[0, :3] = 0
    logits = lin(x)
    logits.retain_grad()
    loss = distill.distill_loss(logits, t, w)
    assert loss.shape == n
    loss.mean().backward()
    wl, wg, _ = head.distill(_np(logits.detach()).reshape(-1, v), host(t.values), host(t.index),
                             host(t.lse) if rest else None, 2.0, host(w).reshape(-1))
    assert np.all(np.abs(host(loss.detach()).reshape(-1) - wl) <= 4.0 * 1.1e-4)
    got = _np(logits.grad).reshape(-1, v)
    # absolute: 1e-4 of w T (q + p) / 24 tokens, bf16 half an ulp (2^-8) more
    tol = 2.0 / 24 * 1e-4 + (2.0 ** -8 * np.abs(wg) / 24 if dtype == "bf16" else 0)
    assert np.all(np.abs(got - wg / 24) <= tol)
    assert lin.weight.grad is not None and torch.isfinite(lin.weight.grad).all()
    assert not got[:3].any()


def test_head_statistics():
    """Two batches through an 8-bit head: loss, covariances, sensitivity."""
    torch.manual_seed(3)
    d, v, k = 128, 512, 24
    W = torch.randn(v, d, device="cuda") * 0.2
    hd = distill.I8Linear.from_weight(W)
    batches, X, G, total = [], [], [], 0.0
    for n, weighted in ((64, False), (40, True)):
        h = (torch.randn(n, d, device="cuda") * torch.exp(torch.randn(d, device="cuda"))).to(torch.bfloat16)
        t = distill.teacher_top(h.float() @ W.t(), k)
        w = (torch.rand(n, device="cuda") > 0.3).float() if weighted else None
        batches.append((h, t, w) if weighted else (h, t))
        logits = hd(h)
        loss, grad = kq.kq_distill_loss_grad(logits, t.values, t.index, t_lse=t.lse, weight=w)
        wl, _, _ = head.distill(_np(logits), host(t.values), host(t.index), host(t.lse), 1.0,
                                None if w is None else host(w))
        np.testing.assert_allclose(host(loss), wl, rtol=0, atol=2e-4)
        total += wl.sum()
        X.append(host(h.view(torch.uint16)))
        G.append(host(grad.view(torch.uint16)))
    st = distill.head_statistics(hd, batches, 104)
    wHX, _, wHG = oracle.covariances(None, np.concatenate(X), np.concatenate(G))
    assert rel_fro(host(st["HX"]), wHX) < 1e-4 and rel_fro(host(st["HG"]), wHG) < 1e-4
    assert abs(st["loss"] - total / 104) < 2e-4
    assert st["loss"] > 0
    want = np.trace(host(st["HX"]).astype(np.float64)) * np.trace(host(st["HG"]).astype(np.float64))
    assert abs(st["s"] / want - 1) < 1e-5
    with pytest.raises(ValueError, match="103"):
        distill.head_statistics(hd, batches, 103)
    with pytest.raises(ValueError, match="104 of 200"):
        distill.head_statistics(hd, batches, 200)


def test_capture_with_the_loss():
    """CovarianceCapture of an inner layer, the divergence from the original
    model's answers as the loss of a coarser copy."""
    torch.manual_seed(4)
    mk = lambda: torch.nn.Sequential(torch.nn.Linear(64, 128), torch.nn.GELU(), torch.nn.Linear(128, 256))
    model = mk().to("cuda", torch.bfloat16)
    with torch.no_grad():
        inp = torch.randn(48, 64, device="cuda").to(torch.bfloat16)
        t = distill.teacher_top(model(inp), 32)
        for p in model.parameters():
            p.add_(torch.randn_like(p) * 0.05)
    layer = model[2]
    seen = []
    h = layer.register_full_backward_hook(lambda m, gi, go: seen.append(go[0].detach()))
    cap = kq.CovarianceCapture(layer, 48)
    with cap.batch():
        distill.distill_loss(model(inp), t).sum().backward()
    HX, D, HG = cap.result()
    cap.remove()
    h.remove()
    _, _, want = oracle.covariances(None, np.zeros((48, 8), np.float32), _np(seen[0]))
    assert rel_fro(host(HG), want) < 1e-4 and np.abs(want).max() > 0

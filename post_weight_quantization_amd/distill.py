"""Layers in 8-bit integers, and the loss that tells what quantization cost:
the divergence from the answers of a teacher (as a rule the model before
quantization), of which only the top logits are kept.

Every step runs in libkq; this module orders the calls and holds the buffers.

  * ``I8Linear`` is a linear layer in 8-bit integers: codes from the sweep
    (``from_codes``) or rounded to nearest (``from_weight``), tokens rounded on
    the way, one token or many.
  * ``teacher_top`` keeps a teacher's answers: the K largest logits of each
    token, their columns, and the log-sum-exp of all.
  * ``distill_loss`` is the loss against them, one value a token, with its
    gradient for torch's autograd: a ``loss_fn`` for ``CovarianceCapture``,
    whose G is then the gradient of the divergence (notes on YAQA, arXiv
    2505.22988: the end-to-end KL).
  * ``head_statistics`` runs the whole of it for the layer that makes the
    logits: 8-bit product, loss, output gradient, covariances, sensitivity.

Usage:
    teacher = teacher_top(model(batch), k=64)            # once, before quantization
    head = I8Linear.from_weight(model.lm_head.weight)
    st = head_statistics(head, [(hidden, teacher)], n_total=hidden.shape[0])
    st["loss"], st["s"]                                  # what it costs; tr(H_G) tr(H_X)
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import api


def _without_gradient(name, t):
    if t is not None and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: expected a tensor that needs no gradient (none is computed for it)")


@dataclass
class I8Linear:
    """y = x W^T + b in 8-bit integers (see kq_linear_i8), in the basis that the
    codes were made in: codes of a layer that ``layer.prepare_layer`` turned
    (incoherence processing) take tokens turned the same way, and give outputs
    in its turned basis; nothing is transformed here."""

    codes: torch.Tensor          # int8, d_out x kq_i8_row_bytes(d_in)
    scale: torch.Tensor          # fp32, d_out
    d_in: int
    zero: torch.Tensor | None = None   # fp32, d_out: zeros of the signed codes
    bias: torch.Tensor | None = None   # fp32, d_out

    @property
    def d_out(self) -> int:
        return self.codes.shape[0]

    @classmethod
    def from_weight(cls, W, bias=None, clip: float = 1.0) -> "I8Linear":
        """Each channel (row of W, bf16 or fp32) rounded to nearest on a
        symmetric grid of its own."""
        codes, scale, _ = api.kq_quantize_rows(W.detach(), clip)
        return cls(codes, scale, W.shape[1], None, None if bias is None else bias.detach().float().contiguous())

    @classmethod
    def from_codes(cls, codes, scale, zero, bias=None) -> "I8Linear":
        """The codes, scales and zeros of kq_gptaq_quantize or kq_yaqa_quantize,
        one grid per channel, any width up to 8 bits."""
        packed, z = api.kq_pack_i8(codes, zero)
        return cls(packed, scale.reshape(-1).contiguous(), codes.shape[1], z,
                   None if bias is None else bias.detach().float().contiguous())

    def __call__(self, x, dtype=None):
        """x: (..., d_in) bf16 or fp32; returns (..., d_out) of x's type, or of
        ``dtype``. Not differentiable: x must not need a gradient, which would be
        lost here (detach it, or call under torch.no_grad())."""
        _without_gradient("x", x)
        y = api.kq_linear_i8(x.detach().reshape(-1, self.d_in), self.codes, self.scale, w_zero=self.zero,
                             bias=self.bias, dtype=dtype)
        return y.reshape(*x.shape[:-1], self.d_out)


@dataclass
class TeacherTop:
    """A teacher's answers to n tokens."""

    values: torch.Tensor         # fp32, n x k: its largest logits
    index: torch.Tensor          # int32, n x k: their columns (below 0: none)
    lse: torch.Tensor | None     # fp32, n: log sum exp(logits / T); None: renormalise over the list
    temperature: float = 1.0


def teacher_top(logits, k: int, temperature: float = 1.0, rest: bool = True) -> TeacherTop:
    """The k largest of logits (..., vocab). rest: keep the log-sum-exp too, so
    that the loss knows the mass off the list."""
    values, index, lse = api.kq_top_logits(logits.detach().reshape(-1, logits.shape[-1]), k, temperature,
                                           want_lse=rest)
    return TeacherTop(values, index, lse, temperature)


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, weight, values, index, lse, temperature):
        loss, stats = api.kq_distill_loss(logits, values, index, lse, temperature, weight)
        ctx.temperature = temperature
        # (all of them, so that torch notices one that was written in between)
        ctx.save_for_backward(logits, weight, values, index, lse, stats)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        logits, weight, values, index, lse, stats = ctx.saved_tensors
        d = (dloss.float() if weight is None else dloss.float() * weight).contiguous()
        grad = api.kq_distill_grad(logits, values, index, stats, d, lse, ctx.temperature)
        return grad, None, None, None, None, None


def distill_loss(logits, teacher: TeacherTop, weight=None):
    """The loss of each token of logits (..., vocab; bf16 or fp32) against the
    teacher's answers, fp32, differentiable in logits. weight: fp32, one a
    token (0: a token that does not count, whatever its logits hold). Neither
    the weights nor the answers may need a gradient, or be written before backward.
    """
    for name, t in (("weight", weight), ("values", teacher.values), ("lse", teacher.lse)):
        _without_gradient(name, t)
    loss = _Distill.apply(logits.reshape(-1, logits.shape[-1]),
                          None if weight is None else weight.reshape(-1).contiguous(), teacher.values,
                          teacher.index, teacher.lse, teacher.temperature)
    return loss.reshape(logits.shape[:-1])


def head_statistics(head: I8Linear, batches, n_total: int) -> dict:
    """Loss and Kronecker statistics of the layer that makes the logits, in 8
    bits, over batches of (hidden, teacher) or (hidden, teacher, weight):
    hidden n x d_in (bf16 or fp32; fp32 with n a multiple of 4), the answers
    to its tokens, and their weights. n_total: tokens of all batches.

    Returns loss (the mean over n_total), HX = X^T X / n_total, HG = G^T G /
    n_total with G the gradient of each token's loss in the layer's output,
    and the sensitivity s with its traces, as kq_sensitivity returns them.
    d_in and the vocabulary must be multiples of 8."""
    seen, losses, HX, HG = 0, [], None, None
    for batch in batches:
        hidden, teacher, weight = batch if len(batch) == 3 else (*batch, None)
        x = hidden.detach().reshape(-1, head.d_in).contiguous()
        logits = head(x)
        loss, G = api.kq_distill_loss_grad(logits, teacher.values, teacher.index, teacher.lse,
                                           teacher.temperature, weight, grad=logits)  # in place of the logits
        losses.append(loss)
        if x.dtype == torch.bfloat16:
            x, G = x.view(torch.uint16), G.view(torch.uint16)
        HX, _, HG = api.kq_accumulate_cov(None, x, G, 1.0 / n_total, 0.0 if seen == 0 else 1.0, HX=HX, HG=HG,
                                          want=("HX", "HG"))
        seen += x.shape[0]
        if seen > n_total:
            raise ValueError(f"{seen} tokens, more than n_total = {n_total}")
    if seen != n_total:
        raise ValueError(f"{seen} of {n_total} tokens seen")
    tx, tg, s = api.kq_sensitivity(HX, HG)
    return dict(loss=float(torch.cat(losses).double().sum()) / n_total, HX=HX, HG=HG, trHX=tx, trHG=tg, s=s)


__all__ = ["I8Linear", "TeacherTop", "teacher_top", "distill_loss", "head_statistics"]

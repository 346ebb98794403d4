"""Thin torch binding of the C ABI in include/kq.h.

Each function has the name of the C entry point it calls and only marshals
arguments: it reads shapes and device pointers from torch tensors, allocates
outputs and scratch memory with torch when the caller passes none, and passes
the current HIP stream. Every step of the computation runs in libkq's kernels.
"""
from __future__ import annotations

import ctypes
import functools

import numpy as np
import torch

from . import _native as N
from ._native import KQError, check  # noqa: F401


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must be on the GPU")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def _expect(t, shape, dtype, name):
    """Shape and dtype of a tensor handed to the library (it sees raw pointers)."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")
    if tuple(t.shape) != tuple(shape) and t.numel() != int(np.prod(shape)):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")


def kq_workspace_size(op: int, d_out: int, d_in: int, n_tok: int = 0, dtype: int = N.KQ_BF16,
                      cfg: N.kq_quant_cfg | None = None) -> int:
    out = ctypes.c_size_t(0)
    check(N.lib.kq_workspace_size(op, d_out, d_in, n_tok, dtype,
                                  ctypes.byref(cfg) if cfg is not None else None, ctypes.byref(out)))
    return out.value


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _ws(nbytes: int, device, ws, stream=None):
    """The caller's workspace, or a new one. A new one is freed when the
    binding returns, possibly with the call's kernels still queued: on a
    stream other than the current one it is recorded there, so the caching
    allocator does not hand it out again before that stream's work is done."""
    if ws is not None:
        return ws
    t = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    if stream is not None and stream != torch.cuda.current_stream(device):
        t.record_stream(stream)
    return t


def kq_accumulate_cov(X, Xq, G, alpha: float, beta: float, HX=None, D=None, HG=None,
                      ws=None, stream=None, want=("HX", "D", "HG")):
    """HX, D, HG <- alpha * (covariance of this chunk) + beta * old (see kq.h).

    X, Xq: (n_tok, d_in); G: (n_tok, d_out); uint16 (bf16 patterns) or float32.
    Outputs listed in ``want`` are allocated when not given.
    """
    ref = Xq if Xq is not None else G
    if ref is None:
        raise ValueError("Xq or G is required")
    if ref.dim() != 2 or ref.dtype not in (torch.float32, torch.uint16, torch.int16, torch.bfloat16):
        raise ValueError(f"inputs must be 2-D float32 or bf16 patterns, got {tuple(ref.shape)} {ref.dtype}")
    dt = N.KQ_F32 if ref.dtype == torch.float32 else N.KQ_BF16
    n_tok = ref.shape[0]
    d_in = Xq.shape[1] if Xq is not None else 8
    d_out = G.shape[1] if G is not None else 8
    f32 = torch.float32
    _expect(X, (n_tok, d_in), ref.dtype, "X")
    _expect(Xq, (n_tok, d_in), ref.dtype, "Xq")
    _expect(G, (n_tok, d_out), ref.dtype, "G")
    _expect(HX, (d_in, d_in), f32, "HX")
    _expect(D, (d_in, d_in), f32, "D")
    _expect(HG, (d_out, d_out), f32, "HG")
    _need_cuda(X, Xq, G, HX, D, HG, ws)
    dev = ref.device
    if HX is None and "HX" in want and Xq is not None:
        HX = torch.empty(d_in, d_in, dtype=torch.float32, device=dev)
    if D is None and "D" in want and X is not None and Xq is not None:
        D = torch.empty(d_in, d_in, dtype=torch.float32, device=dev)
    if HG is None and "HG" in want and G is not None:
        HG = torch.empty(d_out, d_out, dtype=torch.float32, device=dev)
    if ws is None:
        need = kq_workspace_size(N.KQ_OP_ACCUMULATE_COV, d_out, d_in, n_tok, dt)
        ws = _ws(need, dev, None, stream)
    check(N.lib.kq_accumulate_cov(_ptr(X), _ptr(Xq), _ptr(G), dt, n_tok, d_in, d_out, alpha, beta,
                                  _ptr(HX), _ptr(D), _ptr(HG), _ptr(ws), _nbytes(ws), _stream(stream)))
    return HX, D, HG


def kq_biip(W, HX, D, HG, sign_in, sign_out, blk_in: int = 0, blk_out: int = 0, s_x=None,
            s_g=None, ws=None, stream=None):
    """In-place bidirectional incoherence processing; returns (s_x, s_g)."""
    d_out, d_in = W.shape
    f32 = torch.float32
    _expect(W, (d_out, d_in), f32, "W")
    _expect(HX, (d_in, d_in), f32, "HX")
    _expect(D, (d_in, d_in), f32, "D")
    _expect(HG, (d_out, d_out), f32, "HG")
    _expect(sign_in, (d_in,), torch.int8, "sign_in")
    _expect(sign_out, (d_out,), torch.int8, "sign_out")
    _expect(s_x, (d_in,), f32, "s_x")
    _expect(s_g, (d_out,), f32, "s_g")
    _need_cuda(W, HX, D, HG, sign_in, sign_out, s_x, s_g, ws)
    dev = W.device
    if s_x is None:
        s_x = torch.empty(d_in, dtype=torch.float32, device=dev)
    if s_g is None:
        s_g = torch.empty(d_out, dtype=torch.float32, device=dev)
    ws = _ws(kq_workspace_size(N.KQ_OP_BIIP, d_out, d_in), dev, ws, stream)
    check(N.lib.kq_biip(_ptr(W), _ptr(HX), _ptr(D), _ptr(HG), d_out, d_in, _ptr(sign_in),
                        _ptr(sign_out), blk_in, blk_out, _ptr(s_x), _ptr(s_g), _ptr(ws), _nbytes(ws),
                        _stream(stream)))
    return s_x, s_g


def kq_sensitivity(HX, HG, ws=None, stream=None):
    """(tr HX, tr HG, s) as Python floats (synchronizes the stream)."""
    _expect(HX, (HX.shape[0], HX.shape[0]), torch.float32, "HX")
    _expect(HG, (HG.shape[0], HG.shape[0]), torch.float32, "HG")
    _need_cuda(HX, HG, ws)
    ws = _ws(kq_workspace_size(N.KQ_OP_SENSITIVITY, HG.shape[0], HX.shape[0]), HX.device, ws, stream)
    tx, tg, s = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    check(N.lib.kq_sensitivity(_ptr(HX), _ptr(HG), HX.shape[0], HG.shape[0], ctypes.byref(tx),
                               ctypes.byref(tg), ctypes.byref(s), _ptr(ws), _nbytes(ws),
                               _stream(stream)))
    return tx.value, tg.value, s.value


def kq_cholesky_inv(H, damp: float, U=None, ws=None, stream=None):
    """Upper U with U^T U = (H + damp*mean(diag H) I)^-1. Waits for the
    factorization (a non-positive pivot raises); the inverse is left queued
    on the stream."""
    n = H.shape[0]
    _expect(H, (n, n), torch.float32, "H")
    _expect(U, (n, n), torch.float32, "U")
    _need_cuda(H, U, ws)
    if U is None:
        U = torch.empty_like(H)
    ws = _ws(kq_workspace_size(N.KQ_OP_CHOLESKY_INV, n, n), H.device, ws, stream)
    info = ctypes.c_int32(0)
    st = N.lib.kq_cholesky_inv(_ptr(H), n, damp, _ptr(U), ctypes.byref(info), _ptr(ws), _nbytes(ws),
                               _stream(stream))
    check(st, info.value)
    return U


def kq_form_p(D, U, P=None, ws=None, stream=None):
    n = D.shape[0]
    for t, name in ((D, "D"), (U, "U"), (P, "P")):
        _expect(t, (n, n), torch.float32, name)
    _need_cuda(D, U, P, ws)
    if P is None:
        P = torch.empty_like(D)
    ws = _ws(kq_workspace_size(N.KQ_OP_FORM_P, n, n), D.device, ws, stream)
    check(N.lib.kq_form_p(_ptr(D), _ptr(U), n, _ptr(P), _ptr(ws), _nbytes(ws), _stream(stream)))
    return P


def kq_gptaq_quantize(W, U, D, bits: int, group: int = 0, block: int = 128, codes=None,
                      scale=None, zero=None, ws=None, stream=None):
    """In place W0' -> W^'; returns (codes, scale, zero)."""
    d_out, d_in = W.shape
    ng = -(-d_in // group) if group else 1
    f32 = torch.float32
    _expect(W, (d_out, d_in), f32, "W")
    _expect(U, (d_in, d_in), f32, "U")
    _expect(D, (d_in, d_in), f32, "D")
    _expect(codes, (d_out, d_in), torch.uint8, "codes")
    _expect(scale, (d_out, ng), f32, "scale")
    _expect(zero, (d_out, ng), f32, "zero")
    _need_cuda(W, U, D, codes, scale, zero, ws)
    dev = W.device
    cfg = N.kq_quant_cfg(bits, group, block, 0)
    if codes is None:
        codes = torch.empty(d_out, d_in, dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty(d_out, ng, dtype=torch.float32, device=dev)
    if zero is None:
        zero = torch.empty(d_out, ng, dtype=torch.float32, device=dev)
    ws = _ws(kq_workspace_size(N.KQ_OP_GPTAQ_QUANTIZE, d_out, d_in, cfg=cfg), dev, ws, stream)
    check(N.lib.kq_gptaq_quantize(_ptr(W), _ptr(U), _ptr(D), d_out, d_in, ctypes.byref(cfg),
                                  _ptr(codes), _ptr(scale), _ptr(zero), _ptr(ws), _nbytes(ws),
                                  _stream(stream)))
    return codes, scale, zero


def kq_yaqa_quantize(W, U_in, U_out, D, bits: int, codes=None, scale=None, zero=None, ws=None,
                     stream=None):
    """In place W0' -> W^' with feedback along rows (U_in) and columns
    (U_out); returns (codes, scale, zero), one grid per output channel."""
    d_out, d_in = W.shape
    f32 = torch.float32
    _expect(W, (d_out, d_in), f32, "W")
    _expect(U_in, (d_in, d_in), f32, "U_in")
    _expect(U_out, (d_out, d_out), f32, "U_out")
    _expect(D, (d_in, d_in), f32, "D")
    _expect(codes, (d_out, d_in), torch.uint8, "codes")
    _expect(scale, (d_out, 1), f32, "scale")
    _expect(zero, (d_out, 1), f32, "zero")
    _need_cuda(W, U_in, U_out, D, codes, scale, zero, ws)
    dev = W.device
    cfg = N.kq_quant_cfg(bits, 0, 128, 0)
    if codes is None:
        codes = torch.empty(d_out, d_in, dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty(d_out, 1, dtype=torch.float32, device=dev)
    if zero is None:
        zero = torch.empty(d_out, 1, dtype=torch.float32, device=dev)
    ws = _ws(kq_workspace_size(N.KQ_OP_YAQA_QUANTIZE, d_out, d_in, cfg=cfg), dev, ws, stream)
    check(N.lib.kq_yaqa_quantize(_ptr(W), _ptr(U_in), _ptr(U_out), _ptr(D), d_out, d_in,
                                 ctypes.byref(cfg), _ptr(codes), _ptr(scale), _ptr(zero), _ptr(ws),
                                 _nbytes(ws), _stream(stream)))
    return codes, scale, zero


def kq_allocate_bits(s, n_params, widths=(2, 3, 4), avg_budget: float = 2.5):
    L = len(s)
    sa = (ctypes.c_double * L)(*[float(v) for v in s])
    na = (ctypes.c_int64 * L)(*[int(v) for v in n_params])
    wa = (ctypes.c_int32 * len(widths))(*[int(v) for v in widths])
    out = (ctypes.c_int32 * L)()
    check(N.lib.kq_allocate_bits(sa, na, L, wa, len(widths), avg_budget, out))
    return [int(v) for v in out]


def kq_layer_objective(W0, What, HX, D, HG, ws=None, stream=None) -> float:
    d_out, d_in = W0.shape
    f32 = torch.float32
    _expect(W0, (d_out, d_in), f32, "W0")
    _expect(What, (d_out, d_in), f32, "What")
    _expect(HX, (d_in, d_in), f32, "HX")
    _expect(D, (d_in, d_in), f32, "D")
    _expect(HG, (d_out, d_out), f32, "HG")
    _need_cuda(W0, What, HX, D, HG, ws)
    ws = _ws(kq_workspace_size(N.KQ_OP_LAYER_OBJECTIVE, d_out, d_in), W0.device, ws, stream)
    obj = ctypes.c_double()
    check(N.lib.kq_layer_objective(_ptr(W0), _ptr(What), _ptr(HX), _ptr(D), _ptr(HG), d_out, d_in,
                                   ctypes.byref(obj), _ptr(ws), _nbytes(ws), _stream(stream)))
    return obj.value


def kq_set_kernel_events(op: int, start=None, stop=None, stream=None):
    """Bracket the main kernel of later `op` calls on this thread with two
    torch.cuda.Event objects (None, None switches the hook off). The events
    are recorded once here first so that their HIP handles exist."""
    if start is None and stop is None:
        check(N.lib.kq_set_kernel_events(op, None, None))
        return
    s = stream or torch.cuda.current_stream()
    for e in (start, stop):
        if not e.cuda_event:
            e.record(s)
    check(N.lib.kq_set_kernel_events(op, ctypes.c_void_p(start.cuda_event),
                                      ctypes.c_void_p(stop.cuda_event)))


def kq_set_gemm_tile(tile: int) -> None:
    """Force the fp32 product kernel of later calls on this thread: 0 chooses
    by shape (the default), 64, 128 or 256 force that fp32 tile where the
    product allows it, 3 the three-term bf16 kernel wherever it applies. A
    testing knob."""
    check(N.lib.kq_set_gemm_tile(int(tile)))


def kq_packed_row_words(d_in: int, bits: int) -> int:
    out = ctypes.c_int64(0)
    check(N.lib.kq_packed_row_words(d_in, bits, ctypes.byref(out)))
    return out.value


def kq_pack_codes(codes, bits: int, packed=None, stream=None):
    """uint8 codes (d_out x d_in) -> packed 32-bit words, stored as int32 (d_out x row words)."""
    d_out, d_in = codes.shape
    _expect(codes, (d_out, d_in), torch.uint8, "codes")
    if packed is not None:
        _expect(packed, (d_out, kq_packed_row_words(d_in, bits)), packed.dtype, "packed")
        if packed.element_size() != 4:
            raise ValueError("packed: expected 32-bit words")
    _need_cuda(codes, packed)
    if packed is None:
        packed = torch.empty(d_out, kq_packed_row_words(d_in, bits), dtype=torch.int32, device=codes.device)
    check(N.lib.kq_pack_codes(_ptr(codes), d_out, d_in, bits, _ptr(packed), _stream(stream)))
    return packed


def kq_apply_quantized(packed, bits: int, scale, zero, group: int, s_x, s_g, sign_in, sign_out, x,
                       blk_in: int = 0, blk_out: int = 0, y=None, ws=None, stream=None):
    """y = S_G^-1 U^T W^' V S_X^-1 x for x (batch x d_in fp32); returns y (batch x d_out)."""
    batch, d_in = x.shape
    d_out = packed.shape[0]
    f32 = torch.float32
    ng = -(-d_in // group) if group else 1
    _expect(x, (batch, d_in), f32, "x")
    _expect(packed, (d_out, kq_packed_row_words(d_in, bits)), packed.dtype, "packed")
    if packed.element_size() != 4:
        raise ValueError("packed: expected 32-bit words")
    _expect(scale, (d_out, ng), f32, "scale")
    _expect(zero, (d_out, ng), f32, "zero")
    _expect(s_x, (d_in,), f32, "s_x")
    _expect(s_g, (d_out,), f32, "s_g")
    _expect(sign_in, (d_in,), torch.int8, "sign_in")
    _expect(sign_out, (d_out,), torch.int8, "sign_out")
    _expect(y, (batch, d_out), f32, "y")
    _need_cuda(packed, scale, zero, s_x, s_g, sign_in, sign_out, x, y, ws)
    if y is None:
        y = torch.empty(batch, d_out, dtype=torch.float32, device=x.device)
    ws = _ws(kq_workspace_size(N.KQ_OP_APPLY_QUANTIZED, d_out, d_in, batch), x.device, ws, stream)
    check(N.lib.kq_apply_quantized(_ptr(packed), bits, _ptr(scale), _ptr(zero), group, _ptr(s_x),
                                   _ptr(s_g), _ptr(sign_in), _ptr(sign_out), blk_in, blk_out, _ptr(x),
                                   batch, d_out, d_in, _ptr(y), _ptr(ws), _nbytes(ws), _stream(stream)))
    return y


def kq_apply_quantized_noalloc(packed, bits: int, scale, zero, group: int, s_x, s_g, sign_in, sign_out,
                               x, y, blk_in: int = 0, blk_out: int = 0, stream=None):
    """kq_apply_quantized without a workspace: the library's fixed scratch
    array serves instead (for callers that cannot allocate). y (batch x
    d_out fp32) must be given: this call allocates nothing."""
    batch, d_in = x.shape
    d_out = packed.shape[0]
    f32 = torch.float32
    ng = -(-d_in // group) if group else 1
    if y is None:
        raise ValueError("y: expected an output tensor (this call allocates nothing)")
    _expect(x, (batch, d_in), f32, "x")
    _expect(packed, (d_out, kq_packed_row_words(d_in, bits)), packed.dtype, "packed")
    if packed.element_size() != 4:
        raise ValueError("packed: expected 32-bit words")
    _expect(scale, (d_out, ng), f32, "scale")
    _expect(zero, (d_out, ng), f32, "zero")
    _expect(s_x, (d_in,), f32, "s_x")
    _expect(s_g, (d_out,), f32, "s_g")
    _expect(sign_in, (d_in,), torch.int8, "sign_in")
    _expect(sign_out, (d_out,), torch.int8, "sign_out")
    _expect(y, (batch, d_out), f32, "y")
    _need_cuda(packed, scale, zero, s_x, s_g, sign_in, sign_out, x, y)
    check(N.lib.kq_apply_quantized_noalloc(_ptr(packed), bits, _ptr(scale), _ptr(zero), group, _ptr(s_x),
                                           _ptr(s_g), _ptr(sign_in), _ptr(sign_out), blk_in, blk_out,
                                           _ptr(x), batch, d_out, d_in, _ptr(y), _stream(stream)))
    return y


def kq_apply_quantized_a4(packed, scale, zero, s_x, s_g, sign_in, sign_out, x, clip: float = 1.0,
                          blk_in: int = 0, blk_out: int = 0, y=None, act_codes=None, act_scale=None,
                          ws=None, stream=None):
    """The product with 2-bit weights and 4-bit activations: x2 = V S_X^-1 x
    is rounded per vector to s * a (a in [-8, 7], s = clip * max|x2| / 7) and
    y = S_G^-1 U^T W^' (s a). Returns y (batch x d_out); act_codes (batch x
    d_in int8) and act_scale (batch fp32), if given, receive a and s."""
    batch, d_in = x.shape
    d_out = packed.shape[0]
    _expect(x, (batch, d_in), torch.float32, "x")
    _expect(packed, (d_out, kq_packed_row_words(d_in, 2)), packed.dtype, "packed")
    _expect(scale, (d_out,), torch.float32, "scale")
    _expect(zero, (d_out,), torch.float32, "zero")
    _expect(s_x, (d_in,), torch.float32, "s_x")
    _expect(s_g, (d_out,), torch.float32, "s_g")
    _expect(sign_in, (d_in,), torch.int8, "sign_in")
    _expect(sign_out, (d_out,), torch.int8, "sign_out")
    _expect(y, (batch, d_out), torch.float32, "y")
    _expect(act_codes, (batch, d_in), torch.int8, "act_codes")
    _expect(act_scale, (batch,), torch.float32, "act_scale")
    if packed.element_size() != 4:
        raise ValueError("packed: expected 32-bit words")
    _need_cuda(packed, scale, zero, s_x, s_g, sign_in, sign_out, x, y, act_codes, act_scale, ws)
    if y is None:
        y = torch.empty(batch, d_out, dtype=torch.float32, device=x.device)
    ws = _ws(kq_workspace_size(N.KQ_OP_APPLY_QUANTIZED_A4, d_out, d_in, batch), x.device, ws, stream)
    check(N.lib.kq_apply_quantized_a4(_ptr(packed), _ptr(scale), _ptr(zero), _ptr(s_x), _ptr(s_g),
                                      _ptr(sign_in), _ptr(sign_out), blk_in, blk_out, _ptr(x), batch,
                                      d_out, d_in, float(clip), _ptr(y), _ptr(act_codes),
                                      _ptr(act_scale), _ptr(ws), _nbytes(ws), _stream(stream)))
    return y


# ------------------------------------------------- 8-bit product, distillation
_DT = {torch.bfloat16: N.KQ_BF16, torch.float32: N.KQ_F32}


def _raw_stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


@functools.lru_cache(maxsize=1024)
def _need(op, d_out, d_in, n):
    """kq_workspace_size: of the sizes alone, so looked up once for each."""
    return kq_workspace_size(op, d_out, d_in, n)


def _empty(shape, dtype, device, stream):
    """A new tensor in the memory of the stream that the call runs on: no
    earlier work of another stream can still be using that memory."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t, name, cols=None, dtypes=(torch.bfloat16, torch.float32)):
    """(rows, columns, row stride in elements) of a 2-D matrix whose rows may
    lie further apart than they are long."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in dtypes or (
            cols is not None and t.shape[1] != cols):
        want = " or ".join(str(d) for d in dtypes)
        got = f"{tuple(t.shape)} {t.dtype}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: expected a matrix of {want}" +
                         (f" with {cols} columns" if cols is not None else "") + f", got {got}")
    n, m = t.shape
    if m < 1:
        raise ValueError(f"{name}: expected at least one column")
    if m > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: expected rows of adjacent elements, got strides {t.stride()}")
    ld = t.stride(0) if n > 1 else m
    if ld < m:
        raise ValueError(f"{name}: expected rows that do not overlap, got strides {t.stride()}")
    return n, m, ld


def _flat(t, count, dtype, name):
    """A contiguous tensor of `count` elements, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.numel() != count or not t.is_contiguous():
        got = f"{tuple(t.shape)} {t.dtype}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: expected {count} contiguous {dtype}, got {got}")
    return t.data_ptr()


def _on_device(device, *ts):
    if device.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    index = device.index
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors must be on one GPU, got {device} and {t.device}")


def kq_i8_row_bytes(d_in: int) -> int:
    """Bytes of one row of 8-bit codes (d_in padded to a multiple of 128)."""
    out = ctypes.c_int64(0)
    check(N.lib.kq_i8_row_bytes(d_in, ctypes.byref(out)))
    return out.value


def _codes(t, rows, d_in, name):
    rb = (d_in + 127) // 128 * 128
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int8 or t.shape != (rows, rb) or \
            not t.is_contiguous():
        got = f"{tuple(t.shape)} {t.dtype}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: expected contiguous int8 codes {(rows, rb)}, got {got}")
    return t.data_ptr()


def kq_quantize_rows(x, clip: float = 1.0, codes=None, scale=None, sums=None, stream=None):
    """Rows of x (n x d_in, bf16 or fp32) onto symmetric 8-bit grids of their
    own; returns (codes int8 n x row bytes, scale fp32 n, sums int32 n)."""
    n, d, ldx = _rows(x, "x")
    dev = x.device
    _on_device(dev, codes, scale, sums)
    if codes is None:
        codes = _empty((n, kq_i8_row_bytes(d)), torch.int8, dev, stream)
    if scale is None:
        scale = _empty((n,), torch.float32, dev, stream)
    if sums is None:
        sums = _empty((n,), torch.int32, dev, stream)
    check(N.lib.kq_quantize_rows(x.data_ptr(), _DT[x.dtype], n, d, ldx, clip, _codes(codes, n, d, "codes"),
                                 _flat(scale, n, torch.float32, "scale"), _flat(sums, n, torch.int32, "sums"),
                                 _raw_stream(stream, dev)))
    return codes, scale, sums


def kq_pack_i8(codes, zero, packed=None, zero_out=None, stream=None):
    """The sweep's codes (d_out x d_in uint8) and zeros (one per channel) as
    (signed codes int8 d_out x row bytes, zeros fp32 d_out) of the 8-bit product."""
    d_out, d_in = codes.shape
    dev = codes.device
    pc = _flat(codes, d_out * d_in, torch.uint8, "codes")
    pz = _flat(zero, d_out, torch.float32, "zero")
    if pz is None:
        raise ValueError("zero: expected a tensor")
    _on_device(dev, zero, packed, zero_out)
    if packed is None:
        packed = _empty((d_out, kq_i8_row_bytes(d_in)), torch.int8, dev, stream)
    if zero_out is None:
        zero_out = _empty((d_out,), torch.float32, dev, stream)
    check(N.lib.kq_pack_i8(pc, pz, d_out, d_in, _codes(packed, d_out, d_in, "packed"),
                           _flat(zero_out, d_out, torch.float32, "zero_out"), _raw_stream(stream, dev)))
    return packed, zero_out


def _check_out_dtype(y, dtype):
    if y is None and dtype not in _DT:
        raise ValueError(f"dtype: expected torch.bfloat16 or torch.float32, got {dtype}")


def _product_out(y, n, d_out, dtype, dev, stream):
    if y is None:
        y = _empty((n, d_out), dtype, dev, stream)
        return y, d_out
    rows, _, ldy = _rows(y, "y", d_out)
    if rows != n:
        raise ValueError(f"y: expected {n} rows, got {rows}")
    return y, ldy


def kq_matmul_i8(a, a_scale, w, w_scale, d_in: int, a_sum=None, w_zero=None, bias=None, y=None,
                 dtype=torch.bfloat16, ws=None, stream=None):
    """y (n x d_out) = s_t w_o (sum_k a_tk (q_ok - z_o)) + b_o from tokens
    already quantized by kq_quantize_rows. dtype: of y where y is not given."""
    n, d_out = a.shape[0], w.shape[0]
    _check_out_dtype(y, dtype)
    dev = a.device
    _on_device(dev, a_scale, w, w_scale, a_sum, w_zero, bias, y, ws)
    pa, pw = _codes(a, n, d_in, "a"), _codes(w, d_out, d_in, "w")
    f32 = torch.float32
    y, ldy = _product_out(y, n, d_out, dtype, dev, stream)
    if ws is None:
        need = _need(N.KQ_OP_MATMUL_I8, d_out, d_in, n)
        ws = _empty((need,), torch.uint8, dev, stream) if need else None
    check(N.lib.kq_matmul_i8(pa, _flat(a_scale, n, f32, "a_scale"), _flat(a_sum, n, torch.int32, "a_sum"), pw,
                             _flat(w_scale, d_out, f32, "w_scale"), _flat(w_zero, d_out, f32, "w_zero"),
                             _flat(bias, d_out, f32, "bias"), n, d_out, d_in, y.data_ptr(), _DT[y.dtype], ldy,
                             None if ws is None else ws.data_ptr(), 0 if ws is None else _nbytes(ws),
                             _raw_stream(stream, dev)))
    return y


def kq_linear_i8(x, w, w_scale, w_zero=None, bias=None, clip: float = 1.0, y=None, dtype=None, ws=None,
                 stream=None):
    """y (n x d_out) of the 8-bit layer for tokens x (n x d_in, bf16 or fp32):
    kq_quantize_rows and kq_matmul_i8 in one call. dtype: of y where y is not
    given (default: that of x)."""
    n, d_in, ldx = _rows(x, "x")
    d_out = w.shape[0]
    dtype = dtype or x.dtype
    _check_out_dtype(y, dtype)
    dev = x.device
    _on_device(dev, w, w_scale, w_zero, bias, y, ws)
    pw = _codes(w, d_out, d_in, "w")
    f32 = torch.float32
    y, ldy = _product_out(y, n, d_out, dtype, dev, stream)
    if ws is None:
        need = _need(N.KQ_OP_LINEAR_I8, d_out, d_in, n)
        ws = _empty((need,), torch.uint8, dev, stream) if need else None
    check(N.lib.kq_linear_i8(x.data_ptr(), _DT[x.dtype], ldx, clip, pw, _flat(w_scale, d_out, f32, "w_scale"),
                             _flat(w_zero, d_out, f32, "w_zero"), _flat(bias, d_out, f32, "bias"), n, d_out,
                             d_in, y.data_ptr(), _DT[y.dtype], ldy, None if ws is None else ws.data_ptr(),
                             0 if ws is None else _nbytes(ws), _raw_stream(stream, dev)))
    return y


def kq_top_logits(logits, k: int, temperature: float = 1.0, want_lse: bool = True, stream=None):
    """The k largest logits of each row (n x vocab, bf16 or fp32): (values
    fp32 n x k in descending order, index int32 n x k, lse fp32 n of
    logits / temperature, None without want_lse)."""
    n, vocab, ld = _rows(logits, "logits")
    dev = logits.device
    _on_device(dev)
    values = _empty((n, k), torch.float32, dev, stream)
    index = _empty((n, k), torch.int32, dev, stream)
    lse = _empty((n,), torch.float32, dev, stream) if want_lse else None
    check(N.lib.kq_top_logits(logits.data_ptr(), _DT[logits.dtype], n, vocab, ld, k, temperature,
                              values.data_ptr(), index.data_ptr(), lse.data_ptr() if want_lse else None,
                              _raw_stream(stream, dev)))
    return values, index, lse


def _distill_args(logits, values, index, t_lse, temperature, rows, name, *others):
    """The leading arguments that the three distillation calls share."""
    n, vocab, ld = _rows(logits, "logits")
    if not isinstance(values, torch.Tensor) or values.dim() != 2:
        raise ValueError("values: expected a matrix (n x k)")
    k = values.shape[1]
    _on_device(logits.device, values, index, t_lse, rows, *others)
    f32 = torch.float32
    lead = (logits.data_ptr(), _DT[logits.dtype], n, vocab, ld, _flat(values, n * k, f32, "values"),
            _flat(index, n * k, torch.int32, "index"), _flat(t_lse, n, f32, "t_lse"), k, temperature)
    return lead, _flat(rows, n, f32, name)


def _distill_grad_out(logits, grad, stream):
    n, vocab = logits.shape
    if grad is None:
        return _empty((n, vocab), logits.dtype, logits.device, stream), vocab
    rows, _, ldg = _rows(grad, "grad", vocab, (logits.dtype,))
    if rows != n:
        raise ValueError(f"grad: expected {n} rows, got {rows}")
    return grad, ldg


def kq_distill_loss(logits, values, index, t_lse=None, temperature: float = 1.0, weight=None, stream=None):
    """Each row's KL divergence from the teacher's list (kq_top_logits) to the
    student's softmax(logits / T), times weight T^2 (see kq.h). Returns (loss
    fp32 n, stats fp32 n x 3 for kq_distill_grad)."""
    lead, pw = _distill_args(logits, values, index, t_lse, temperature, weight, "weight")
    n, dev = logits.shape[0], logits.device
    loss = _empty((n,), torch.float32, dev, stream)
    stats = _empty((n, 3), torch.float32, dev, stream)
    check(N.lib.kq_distill_loss(*lead, pw, loss.data_ptr(), stats.data_ptr(), _raw_stream(stream, dev)))
    return loss, stats


def kq_distill_grad(logits, values, index, stats, dloss, t_lse=None, temperature: float = 1.0, grad=None,
                    stream=None):
    """The gradient in the logits, given the forward call's stats and the
    gradient dloss (n) of its losses. grad may be the logits themselves."""
    lead, pd = _distill_args(logits, values, index, t_lse, temperature, dloss, "dloss", stats, grad)
    if pd is None:
        raise ValueError("dloss: expected a tensor")
    n, dev = logits.shape[0], logits.device
    ps = _flat(stats, 3 * n, torch.float32, "stats")
    grad, ldg = _distill_grad_out(logits, grad, stream)
    check(N.lib.kq_distill_grad(*lead, ps, pd, grad.data_ptr(), ldg, _raw_stream(stream, dev)))
    return grad


def kq_distill_loss_grad(logits, values, index, t_lse=None, temperature: float = 1.0, weight=None, grad=None,
                         stream=None):
    """(loss n, gradient n x vocab of the sum of the losses) in one pass. grad
    may be the logits themselves."""
    lead, pw = _distill_args(logits, values, index, t_lse, temperature, weight, "weight", grad)
    n, dev = logits.shape[0], logits.device
    loss = _empty((n,), torch.float32, dev, stream)
    grad, ldg = _distill_grad_out(logits, grad, stream)
    check(N.lib.kq_distill_loss_grad(*lead, pw, loss.data_ptr(), None, grad.data_ptr(), ldg,
                                     _raw_stream(stream, dev)))
    return loss, grad

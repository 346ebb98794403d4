"""Every argument check of the 8-bit product, the top logits and the
distillation loss, one case each (CPU): rejected on the host, before any
launch, with the status the header documents."""
import ctypes
import math
import os
import re

import pytest

N = pytest.importorskip("post_weight_quantization_amd._native")


def _gpu_present():
    try:
        import torch
        return torch.cuda.device_count() > 0
    except Exception:  # pragma: no cover
        return False


# a fake device pointer must never reach a launch on a real device
pytestmark = pytest.mark.skipif(_gpu_present(), reason="fake device pointers: host-only checks")

A, B, C, ODD = 0x100000, 0x200000, 0x300000, 0x100003
BIG = 1 << 50
ARG, SHAPE, WS, UNS = N.KQ_ERR_ARG, N.KQ_ERR_SHAPE, N.KQ_ERR_WORKSPACE, N.KQ_ERR_UNSUPPORTED


def rowb(d_in=10, out=True):
    b = ctypes.c_int64()
    return N.lib.kq_i8_row_bytes(d_in, ctypes.byref(b) if out else None)


def quant(x=A, dt=N.KQ_BF16, n=4, d=64, ldx=64, clip=1.0, codes=B, scale=C, sums=C):
    return N.lib.kq_quantize_rows(x, dt, n, d, ldx, clip, codes, scale, sums, None)


def pack(codes=A, zero=B, m=4, d=8, packed=C, zo=B):
    return N.lib.kq_pack_i8(codes, zero, m, d, packed, zo, None)


def mm(a=A, s=B, asum=C, w=A, ws_=B, wz=None, n=4, m=16, d=64, y=C, dt=N.KQ_F32, ldy=16, ws=C, wsb=BIG):
    return N.lib.kq_matmul_i8(a, s, asum, w, ws_, wz, None, n, m, d, y, dt, ldy, ws, wsb, None)


def lin(x=A, dt=N.KQ_BF16, ldx=64, clip=1.0, w=A, ws_=B, n=4, m=16, d=64, y=C, ydt=N.KQ_F32, ldy=16, ws=C,
        wsb=BIG):
    return N.lib.kq_linear_i8(x, dt, ldx, clip, w, ws_, None, None, n, m, d, y, ydt, ldy, ws, wsb, None)


def top(x=A, dt=N.KQ_BF16, n=4, v=100, ld=100, k=5, t=1.0, val=B, idx=C):
    return N.lib.kq_top_logits(x, dt, n, v, ld, k, t, val, idx, None, None)


def loss(x=A, dt=N.KQ_BF16, n=4, v=100, ld=100, val=B, idx=C, k=5, t=1.0, out=B):
    return N.lib.kq_distill_loss(x, dt, n, v, ld, val, idx, None, k, t, None, out, None, None)


def grad(x=A, dt=N.KQ_BF16, n=4, v=100, ld=100, val=B, idx=C, k=5, t=1.0, stats=B, dl=B, g=C, ldg=100):
    return N.lib.kq_distill_grad(x, dt, n, v, ld, val, idx, None, k, t, stats, dl, g, ldg, None)


def both(x=A, dt=N.KQ_BF16, n=4, v=100, ld=100, val=B, idx=C, k=5, t=1.0, out=B, g=C, ldg=100):
    return N.lib.kq_distill_loss_grad(x, dt, n, v, ld, val, idx, None, k, t, None, out, None, g, ldg, None)


def wsize(op, m=8, d=8, n=4):
    b = ctypes.c_size_t()
    return N.lib.kq_workspace_size(op, m, d, n, 0, None, ctypes.byref(b))


CASES = [
    ("row bytes null", lambda: rowb(out=False), ARG, "NULL"),
    ("row bytes 0", lambda: rowb(0), SHAPE, "d_in"),
    ("row bytes too many", lambda: rowb(65537), SHAPE, "65536"),
    ("quant tokens", lambda: quant(n=-1), SHAPE, "n_tok"),
    ("quant too many tokens", lambda: quant(n=1048577), SHAPE, "1048576"),
    ("quant d_in 0", lambda: quant(d=0), SHAPE, "d_in"),
    ("quant d_in large", lambda: quant(d=65537, ldx=70000), SHAPE, "65536"),
    ("quant dtype", lambda: quant(dt=5), ARG, "dtype"),
    ("quant clip 0", lambda: quant(clip=0.0), ARG, "clip"),
    ("quant clip nan", lambda: quant(clip=math.nan), ARG, "clip"),
    ("quant clip above 1", lambda: quant(clip=1.01), ARG, "clip"),
    ("quant ldx", lambda: quant(ldx=63), SHAPE, "ldx"),
    ("quant null x", lambda: quant(x=None), ARG, "NULL"),
    ("quant null sums", lambda: quant(sums=None), ARG, "NULL"),
    ("quant odd x", lambda: quant(x=ODD), ARG, "aligned to its type"),
    ("quant odd codes", lambda: quant(codes=B + 8), ARG, "16-byte"),
    ("pack null", lambda: pack(zero=None), ARG, "NULL"),
    ("pack d_out", lambda: pack(m=0), SHAPE, "d_out"),
    ("pack d_in", lambda: pack(d=0), SHAPE, "d_in"),
    ("pack odd", lambda: pack(packed=C + 4), ARG, "16-byte"),
    ("matmul tokens", lambda: mm(n=-2), SHAPE, "n_tok"),
    ("matmul d_out", lambda: mm(m=1048577, ldy=1 << 21), SHAPE, "d_out"),
    ("matmul null w", lambda: mm(w=None), ARG, "NULL"),
    ("matmul dtype", lambda: mm(dt=2), ARG, "dtype"),
    ("matmul ldy", lambda: mm(ldy=15), SHAPE, "ldy"),
    ("matmul odd w", lambda: mm(w=A + 8), ARG, "16-byte"),
    ("matmul odd y", lambda: mm(y=C + 2), ARG, "aligned to its type"),
    ("matmul null a", lambda: mm(a=None), ARG, "NULL"),
    ("matmul zeros without sums", lambda: mm(wz=B, asum=None), ARG, "a_sum"),
    ("matmul odd a", lambda: mm(a=ODD), ARG, "16-byte"),
    ("linear dtype", lambda: lin(dt=9), ARG, "dtype"),
    ("linear clip", lambda: lin(clip=-1.0), ARG, "clip"),
    ("linear ldx", lambda: lin(ldx=10), SHAPE, "ldx"),
    ("linear null x", lambda: lin(x=None), ARG, "NULL"),
    ("linear null y", lambda: lin(y=None), ARG, "NULL"),
    ("linear odd x", lambda: lin(x=ODD), ARG, "aligned to its type"),
    ("linear no workspace", lambda: lin(n=40, ws=None), WS, "required"),
    ("linear small workspace", lambda: lin(n=40, wsb=16), WS, "required"),
    ("linear odd workspace", lambda: lin(n=40, ws=C + 8), ARG, "workspace must be 16-byte"),
    ("top dtype", lambda: top(dt=3), ARG, "dtype"),
    ("top rows", lambda: top(n=-1), SHAPE, "0 <= n"),
    ("top ld", lambda: top(ld=99), SHAPE, "vocab <= ld"),
    ("top vocab 0", lambda: top(v=0), SHAPE, "vocab"),
    ("top k 0", lambda: top(k=0), SHAPE, "k"),
    ("top k 257", lambda: top(k=257, v=1000, ld=1000), SHAPE, "256"),
    ("top k above vocab", lambda: top(k=101), SHAPE, "k <= vocab"),
    ("top vocab above int32", lambda: top(v=1 << 31, ld=1 << 31), SHAPE, "2^30"),
    ("top temperature 0", lambda: top(t=0.0), ARG, "temperature"),
    ("top temperature inf", lambda: top(t=math.inf), ARG, "temperature"),
    ("top null", lambda: top(idx=None), ARG, "NULL"),
    ("top odd", lambda: top(x=ODD), ARG, "aligned"),
    ("loss vocab", lambda: loss(v=524289, ld=524289), UNS, "524288"),
    ("loss temperature", lambda: loss(t=math.nan), ARG, "temperature"),
    ("loss null list", lambda: loss(idx=None), ARG, "NULL"),
    ("loss odd", lambda: loss(x=ODD), ARG, "aligned"),
    ("loss null out", lambda: loss(out=None), ARG, "NULL"),
    ("grad null stats", lambda: grad(stats=None), ARG, "NULL"),
    ("grad null grad", lambda: grad(g=None), ARG, "NULL"),
    ("grad ldg", lambda: grad(ldg=99), SHAPE, "ldg"),
    ("grad in place with another stride", lambda: grad(g=A, ldg=128), ARG, "in place"),
    ("grad odd", lambda: grad(g=ODD), ARG, "aligned"),
    ("both null loss", lambda: both(out=None), ARG, "NULL"),
    ("both null grad", lambda: both(g=None), ARG, "NULL"),
    ("wsize matmul", lambda: wsize(N.KQ_OP_MATMUL_I8, n=-1), SHAPE, "sizes"),
    ("wsize linear", lambda: wsize(N.KQ_OP_LINEAR_I8, m=0), SHAPE, "sizes"),
]


@pytest.mark.parametrize("name,call,status,words", CASES, ids=[c[0] for c in CASES])
def test_rejected_on_the_host(name, call, status, words):
    st = call()
    msg = N.lib.kq_last_error().decode()
    assert N.STATUS_NAMES.get(st) == N.STATUS_NAMES[status], (name, st, msg)
    assert words in msg, (name, msg)


def test_the_table_reaches_every_check():
    src = open(os.path.join(os.path.dirname(N.__file__), "csrc", "kq_api_head.hip")).read()
    msgs = set(re.findall(r'fail\(KQ_ERR_\w+,\s*"([^"]+)"', src))
    reached = set()
    for _, call, _, _ in CASES:
        call()
        reached.add(N.lib.kq_last_error().decode())
    missing = []
    for m in sorted(msgs):
        pat = re.escape(re.sub(r"%(?:zu|lld|d|s)", "\x00", m)).replace("\x00", ".*")
        if not any(re.match(pat, r) for r in reached):
            missing.append(m)
    assert not missing, missing


def test_nothing_to_do_is_not_an_error():
    """No tokens or rows: accepted without a pointer."""
    assert quant(x=None, n=0, codes=None, scale=None, sums=None) == N.KQ_OK
    assert mm(a=None, s=None, w=None, ws_=None, n=0, y=None, ws=None, wsb=0) == N.KQ_OK
    assert lin(x=None, w=None, n=0, y=None, ws=None, wsb=0) == N.KQ_OK
    assert top(x=None, n=0, val=None, idx=None) == N.KQ_OK
    assert loss(x=None, n=0, val=None, idx=None, out=None) == N.KQ_OK
    assert grad(x=None, n=0, val=None, idx=None, stats=None, dl=None, g=None) == N.KQ_OK
    assert both(x=None, n=0, val=None, idx=None, out=None, g=None) == N.KQ_OK
    assert wsize(N.KQ_OP_LINEAR_I8, n=0) == N.KQ_OK


@pytest.mark.parametrize("m,d,n", [(16, 64, 40), (300, 1001, 700), (8192, 28672, 12), (4096, 4096, 5), (256, 28672, 3), (8192, 28672, 64)])
def test_workspace_one_byte_short(m, d, n):
    b = ctypes.c_size_t()
    for op, call in ((N.KQ_OP_LINEAR_I8, lin), (N.KQ_OP_MATMUL_I8, mm)):
        assert N.lib.kq_workspace_size(op, m, d, n, 0, None, ctypes.byref(b)) == N.KQ_OK
        if b.value:
            kw = dict(ldx=d) if call is lin else {}
            assert call(m=m, d=d, n=n, ldy=m, wsb=b.value - 1, **kw) == N.KQ_ERR_WORKSPACE
            assert str(b.value) in N.lib.kq_last_error().decode()


def test_bindings_reject_wrong_tensors():
    import torch

    from post_weight_quantization_amd import api

    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    i8, i32 = torch.int8, torch.int32
    cases = [
        ("x", lambda: api.kq_quantize_rows(z(4, 8, dt=torch.float64))),
        ("x", lambda: api.kq_quantize_rows(z(8))),
        ("x", lambda: api.kq_quantize_rows(z(8, 4).t())),
        ("x", lambda: api.kq_quantize_rows(z(1, 8).expand(4, 8))),
        ("codes", lambda: api.kq_pack_i8(z(4, 8), z(4))),
        ("zero", lambda: api.kq_pack_i8(z(4, 8, dt=torch.uint8), z(5))),
        ("logits", lambda: api.kq_top_logits(z(4, 8, dt=torch.float16), 2)),
        ("logits", lambda: api.kq_distill_loss(z(4), z(4, 2), z(4, 2, dt=i32))),
        ("values", lambda: api.kq_distill_loss(z(4, 9), z(4), z(4, dt=i32))),
    ]
    for name, call in cases:
        with pytest.raises(ValueError, match=rf"^{name}: expected"):
            call()
    # the rest is looked at once the tensors are known to be on a GPU
    for call in (lambda: api.kq_linear_i8(z(4, 8), z(3, 128, dt=i8), z(3)),
                 lambda: api.kq_matmul_i8(z(4, 128, dt=i8), z(4), z(3, 128, dt=i8), z(3), 8),
                 lambda: api.kq_top_logits(z(4, 8), 2),
                 lambda: api.kq_distill_loss_grad(z(4, 9), z(4, 2), z(4, 2, dt=i32))):
        with pytest.raises(ValueError, match="GPU"):
            call()

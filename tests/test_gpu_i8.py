"""GPU parity of the 8-bit product (kq_quantize_rows, kq_pack_i8,
kq_matmul_i8, kq_linear_i8) against oracle/head.py.

Codes, scales and code sums are decided in fp32 by the same correctly rounded
operations on both sides, so they are compared for equality. The product's
sum is an exact integer; what follows rounds: int32 -> fp32, two products and
the bias, half an ulp (2^-24) each, so fp32 outputs lie within 4 * 2^-24 of
|y - b| + |b|, and a bf16 output between the roundings of both ends of that
range.
"""
import numpy as np
import pytest

from oracle import head
from tests.gpu_util import bf16, have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

if have_gpu():
    import torch

    import post_weight_quantization_amd as kq


def _tokens(n, d, dtype, seed, stride=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, d, device="cuda", generator=g) * torch.exp(torch.randn(d, device="cuda", generator=g))
    buf = torch.full((n, d + stride), float("nan"), dtype=dtype, device="cuda")
    buf[:, :d] = x.to(dtype)
    return buf[:, :d]


def _weights(m, d, seed, low=-128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.zeros(m, kq.kq_i8_row_bytes(d), dtype=torch.int8, device="cuda")
    w[:, :d] = torch.randint(low, 128, (m, d), device="cuda", generator=g).to(torch.int8)
    scale = torch.rand(m, device="cuda", generator=g) * 0.01 + 1e-4
    zero = torch.randint(-128, 128, (m,), device="cuda", generator=g).float()
    bias = torch.randn(m, device="cuda", generator=g)
    return w, scale, zero, bias


def _np(t):
    return host(t.float()) if t.dtype == torch.bfloat16 else host(t)


def _check(y, want, bias, dtype):
    b = 0.0 if bias is None else np.abs(host(bias).astype(np.float64))[None, :]
    tol = 4 * 2.0 ** -24 * (np.abs(want) + 2 * b) + 1e-37
    lo, hi = want - tol, want + tol
    if dtype == torch.bfloat16:
        lo, hi = bf16(lo), bf16(hi)
    got = _np(y).astype(np.float64)
    bad = ~((lo <= got) & (got <= hi))
    assert not bad.any(), (int(bad.sum()), got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,stride", [(1, 1, 0), (3, 7, 5), (2, 128, 0), (5, 1001, 3), (4, 4096, 0),
                                        (2, 28672, 8), (1, 65536, 0), (300, 640, 1)])
def test_quantize_rows_exact(n, d, stride, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = _tokens(n, d, dt, n + d, stride)
    for clip in (1.0, 0.9):
        codes, scale, sums = kq.kq_quantize_rows(x, clip)
        c, s, t = head.quantize_rows(_np(x), clip)
        np.testing.assert_array_equal(host(scale), s)
        np.testing.assert_array_equal(host(codes)[:, :d], c)
        assert not host(codes)[:, d:].any()
        np.testing.assert_array_equal(host(sums), t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_rows_that_are_not_ordinary(dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = _tokens(9, 300, dt, 5).contiguous()
    x[0] = 0.0
    x[1, 299] = float("nan")
    x[2, 0] = float("inf")
    x[3, 17] = float("-inf")
    x[4] *= 1e-36
    x[5] = 0.0
    x[5, 3] = 1e-45 if dt == torch.float32 else 1e-40   # a scale that underflows or is denormal
    x[6] *= 1e36
    x[7] = -0.0
    codes, scale, sums = kq.kq_quantize_rows(x)
    c, s, t = head.quantize_rows(_np(x))
    np.testing.assert_array_equal(host(scale), s)
    np.testing.assert_array_equal(host(codes)[:, :300], c)
    np.testing.assert_array_equal(host(sums), t)
    w, ws, _, _ = _weights(40, 300, 1)
    y = kq.kq_linear_i8(x, w, ws)
    assert torch.isnan(y[1:4]).all() and not torch.isnan(y[4:]).any()
    assert not y[0].any() and not y[7].any()


# one token; few tokens; tiles cut on both sides; K of one byte, of several
# tiles and of an odd length; many tokens (the widest tiles, ragged)
SHAPES = [(1, 1, 1), (1, 64, 4096), (1, 4096, 128), (2, 100, 300), (7, 2777, 1001), (15, 512, 2048),
          (16, 130, 8192), (17, 96, 640), (33, 257, 129), (64, 1000, 4096), (100, 4097, 1024),
          (129, 255, 513), (300, 1024, 4096), (513, 1027, 777), (1500, 2050, 1100), (4100, 520, 256),
          (40, 16, 65536), (4, 300, 28672), (24, 8192, 1024), (2048, 2816, 640),
          # each tile, and each with K shared
          (276, 27058, 68), (1030, 8200, 1000), (4129, 65, 16113), (2000, 10900, 500), (68, 4192, 11572),
          (140, 23126, 64), (4155, 67, 8009),
          (65, 2238, 15982), (40, 260, 30000), (600, 600, 20000),
          # few tokens, kept in registers (1, 2 lines of each of 8, 16 waves; shared) and not (long rows shared)
          (7, 11000, 1000), (20, 16400, 400), (3, 10500, 1500), (31, 10300, 2000), (10, 10300, 3000),
          (30, 12000, 4096), (16, 4100, 11000), (30, 4100, 6000), (30, 9000, 3000), (9, 1000, 20000),
          (4, 1000, 4096), (3, 12000, 4000)]


@pytest.mark.parametrize("n,m,d", SHAPES)
def test_linear_against_oracle(n, m, d):
    print(f"[i8] {n} x {d} -> {m}", flush=True)
    w, scale, zero, bias = _weights(m, d, m + d)
    for dt, z, b, stride in ((torch.bfloat16, None, None, 0), (torch.float32, zero, bias, 3),
                             (torch.bfloat16, zero, None, 1)):
        x = _tokens(n, d, dt, n + m, stride)
        y = kq.kq_linear_i8(x, w, scale, w_zero=z, bias=b)
        c, s, _ = head.quantize_rows(_np(x))
        want, _ = head.product(c, s, host(w)[:, :d], host(scale), None if z is None else host(z),
                               None if b is None else host(b))
        assert y.dtype == dt
        _check(y, want, b, dt)


@pytest.mark.parametrize("n,m,d", [(1, 96, 1024), (5, 33, 700), (20, 200, 1024), (130, 140, 999),
                                   (600, 700, 1024)])
def test_product_bit_exact(n, m, d):
    """Unit scales and small codes: y is the integer sum itself."""
    g = torch.Generator(device="cuda").manual_seed(d)
    rb = kq.kq_i8_row_bytes(d)
    a = torch.zeros(n, rb, dtype=torch.int8, device="cuda")
    a[:, :d] = torch.randint(-127, 128, (n, d), device="cuda", generator=g).to(torch.int8)
    w, _, zero, _ = _weights(m, d, d)
    one = lambda k: torch.ones(k, device="cuda")
    sums = a.sum(1).to(torch.int32)
    y = kq.kq_matmul_i8(a, one(n), w, one(m), d, a_sum=sums, w_zero=zero, dtype=torch.float32)
    _, acc = head.product(host(a)[:, :d].astype(np.int64), np.ones(n, np.float32), host(w)[:, :d],
                          np.ones(m), host(zero))
    assert np.abs(acc).max() < 2 ** 31
    np.testing.assert_array_equal(host(y), acc.astype(np.float32))


def test_product_at_the_int32_edge():
    """The largest sums: d_in = 65536 of codes 127 against -128 - 127."""
    d = 65536
    a = torch.full((2, d), 127, dtype=torch.int8, device="cuda")
    a[1] = -127
    w = torch.full((20, d), -128, dtype=torch.int8, device="cuda")
    sums = a.sum(1, dtype=torch.int64).to(torch.int32)
    y = kq.kq_matmul_i8(a, torch.ones(2, device="cuda"), w, torch.ones(20, device="cuda"), d, a_sum=sums,
                        w_zero=torch.full((20,), 127.0, device="cuda"), dtype=torch.float32)
    want = np.float32(-127 * 255 * d)
    np.testing.assert_array_equal(host(y), np.stack([np.full(20, want), np.full(20, -want)]))


def test_pack_of_the_sweeps_codes():
    g = torch.Generator(device="cuda").manual_seed(2)
    for bits, d in ((8, 333), (2, 128), (4, 1)):
        codes = torch.randint(0, 1 << bits, (37, d), device="cuda", generator=g).to(torch.uint8)
        zero = torch.randint(0, 1 << bits, (37, 1), device="cuda", generator=g).float()
        packed, z = kq.kq_pack_i8(codes, zero)
        assert packed.shape == (37, kq.kq_i8_row_bytes(d))
        np.testing.assert_array_equal(host(packed)[:, :d].astype(int), host(codes).astype(int) - 128)
        assert not host(packed)[:, d:].any()
        np.testing.assert_array_equal(host(z), host(zero)[:, 0] - 128)
        # w = scale (q - zero), whichever way it is stored
        x = _tokens(3, d, torch.float32, d)
        scale = torch.rand(37, device="cuda", generator=g)
        y = kq.kq_linear_i8(x, packed, scale, w_zero=z)
        c, s, _ = head.quantize_rows(_np(x))
        want, _ = head.product(c, s, host(codes).astype(int), host(scale), host(zero)[:, 0])
        _check(y, want, None, torch.float32)


@pytest.mark.parametrize("n", [1, 9, 200])
def test_output_rows_of_their_own_stride(n):
    m, d = 70, 260
    w, scale, _, _ = _weights(m, d, 4)
    x = _tokens(n, d, torch.float32, 8)
    buf = torch.full((n, m + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    kq.kq_linear_i8(x, w, scale, y=buf[:, :m])
    c, s, _ = head.quantize_rows(_np(x))
    want, _ = head.product(c, s, host(w)[:, :d], host(scale))
    _check(buf[:, :m], want, None, torch.bfloat16)
    assert (buf[:, m:] == 7.0).all()


def test_no_tokens():
    w, scale, _, _ = _weights(10, 20, 0)
    y = kq.kq_linear_i8(torch.empty(0, 20, device="cuda"), w, scale)
    assert y.shape == (0, 10)
    codes, s, t = kq.kq_quantize_rows(torch.empty(0, 20, device="cuda"))
    assert kq.kq_matmul_i8(codes, s, w, scale, 20, a_sum=t).shape == (0, 10)


@pytest.mark.parametrize("n", [1, 40, 700])
def test_repeat_calls_another_stream_and_graph(n):
    """The same bits on every call, on a stream of the caller's, and from
    replays of a graph with other work between them."""
    m, d = 1030, 2000
    w, scale, zero, bias = _weights(m, d, 6)
    x = _tokens(n, d, torch.bfloat16, 7, 3)
    kw = dict(w_zero=zero, bias=bias)
    y = kq.kq_linear_i8(x, w, scale, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2 = kq.kq_linear_i8(x, w, scale, stream=side, **kw)
    side.synchronize()
    assert torch.equal(y, y2)
    static = x.clone()
    out = torch.empty(n, m, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kq.kq_workspace_size(kq._native.KQ_OP_LINEAR_I8, m, d, n), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kq.kq_linear_i8(static, w, scale, y=out, ws=ws, **kw)
    for rep in range(3):
        static.copy_(x * (rep + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kq.kq_linear_i8(static, w, scale, **kw)), rep


@pytest.mark.slow
@pytest.mark.parametrize("n,m,d", [(1, 8192, 28672), (12, 8192, 28672), (2048, 11008, 4096), (4096, 8192, 28672)])
def test_full_size(n, m, d):
    """Sampled tokens and channels of the full-size products, exactly."""
    print(f"[i8 full] {n} x {d} -> {m}", flush=True)
    w, scale, zero, _ = _weights(m, d, 9)
    x = _tokens(n, d, torch.bfloat16, 10)
    y = kq.kq_linear_i8(x, w, scale, w_zero=zero, dtype=torch.float32)
    rng = np.random.default_rng(0)
    ti = np.unique(np.r_[0, n - 1, rng.integers(0, n, 60)])
    oi = np.unique(np.r_[0, m - 1, rng.integers(0, m, 200)])
    ti_t, oi_t = torch.from_numpy(ti).cuda(), torch.from_numpy(oi).cuda()
    c, s, _ = head.quantize_rows(_np(x[ti_t]))
    want, _ = head.product(c, s, host(w[oi_t])[:, :d], host(scale[oi_t]), host(zero[oi_t]))
    got = host(y[ti_t][:, oi_t]).astype(np.float64)
    assert np.all(np.abs(got - want) <= 4 * 2.0 ** -24 * np.abs(want))

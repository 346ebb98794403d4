"""GPU parity of the teacher's top logits and of the distillation loss and
gradient against oracle/head.py.

Top logits: values and indices are compared for equality. Their log-sum-exp,
and the losses, come from fp32 sums of exponentials. An exponential of x is
off by 2^-23 (1 + |x|) relative (its own ulp, and the rounding of the scaled
argument); weighted with the exponentials themselves |x| averages at most
log(vocab) <= 13.2, and a sum of up to 525 values a thread and 10 joining steps adds
at most 535 * 2^-24 in the worst order: below 4e-5 together. So
  lse    within 4e-5 + 2^-22 |lse| (its own rounding),
  loss   within w T^2 (1e-4 P + 2^-22 max|z|): the sum and the mass off the
         list both enter (4e-5 each), and z = (s - max) / T is rounded,
  grad   within w T 1e-4 (q (P + r / q_r) + p): q, and r / q_r, carry the
         same errors, q also the rounding of s / T - lse (2^-23 times up to 100);
         a bf16 gradient lies between the roundings of both ends of that range.
"""
import numpy as np
import pytest

from oracle import head
from tests.gpu_util import bf16, have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

if have_gpu():
    import torch

    import post_weight_quantization_amd as kq

DT = {"bf16": "bfloat16", "f32": "float32"}
INF = float("inf")


def _np(t):
    return host(t.float()) if t.dtype == torch.bfloat16 else host(t)


def _logits(n, v, dtype, seed, stride=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(n, v, device="cuda", generator=g) * spread
    buf = torch.full((n, v + stride), float("nan"), dtype=getattr(torch, DT[dtype]), device="cuda")
    buf[:, :v] = t
    return buf[:, :v]


def _check_top(logits, k, temperature=1.0):
    v, i, lse = kq.kq_top_logits(logits, k, temperature)
    wv, wi, wl = head.top_logits(_np(logits), k, temperature)
    np.testing.assert_array_equal(host(i), wi)
    np.testing.assert_array_equal(host(v), wv.astype(np.float32))
    with np.errstate(invalid="ignore", over="ignore"):  # a sum past fp32 is inf
        ok = (np.abs(host(lse) - wl) <= 4e-5 + 2.0 ** -22 * np.abs(wl)) | (host(lse) == wl.astype(np.float32)) | \
             (np.isnan(host(lse)) & np.isnan(wl))
    assert ok.all(), (host(lse), wl)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,k,stride", [(1, 1, 1, 0), (3, 7, 7, 2), (2, 256, 256, 0), (5, 1000, 10, 1),
                                          (4, 1025, 256, 7), (3, 32000, 64, 0), (2, 50001, 200, 3),
                                          (9, 8191, 1, 0), (1, 128256, 64, 0), (2, 164001, 33, 0),
                                          (300, 517, 5, 0), (1, 530000, 100, 5), (270, 16385, 40, 1)])
def test_top_logits(n, v, k, stride, dtype):
    print(f"[top] {n} x {v} k {k} {dtype}", flush=True)
    _check_top(_logits(n, v, dtype, n + v, stride), k, 1.0 if k % 2 else 0.7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [600, 33333, 100000])
def test_top_logits_ties_and_order(v, dtype):
    """Equal logits everywhere, few distinct values, ascending and descending
    rows, one spike, everything in one corner."""
    rng = np.random.default_rng(v)
    rows = [np.zeros(v), rng.integers(0, 3, v), np.arange(v) / 64.0, -np.arange(v) / 64.0,
            np.r_[np.zeros(v - 1), 1.0], np.r_[rng.normal(5, 1, 300), np.full(v - 300, -4.0)],
            np.where(rng.random(v) < 0.5, 0.0, -0.0), np.full(v, -INF)]
    t = torch.tensor(np.array(rows), dtype=torch.float32, device="cuda").to(getattr(torch, DT[dtype]))
    for k in (1, 64, 256):
        _check_top(t, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_top_logits_masked_and_not_finite(dtype):
    t = _logits(8, 3000, dtype, 4).contiguous()
    low = torch.finfo(t.dtype).min
    t[0, 5:] = -INF               # five left, fewer than k
    t[1, :] = -INF                # none left
    t[2, 10:] = low               # a mask of the type's lowest value
    t[3, :] = low
    t[4, 100] = float("nan")
    t[4, 2000] = float("nan")
    t[5, 7] = INF
    t[6, 0::2] = -INF
    _check_top(t, 20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [1e-4, 1.0, 300.0])
def test_top_logits_of_any_magnitude(temperature, dtype):
    """Rows far from zero, up to the type's largest numbers of either sign, and
    temperatures that take logits / T past them. The bound of the other tests:
    m / T in three roundings, 2^-22 of it; the logarithm of the sum, terms of
    which count down to 2^-25, within 25 * 2^-23 and the sum's own roundings."""
    top = torch.finfo(getattr(torch, DT[dtype])).max
    offsets = [0.0, 30.0, -2000.0, 1e5, -7e8, 8e8, 1e20, 0.5 * top, -0.5 * top]
    rng = np.random.default_rng(3)
    t = torch.tensor(np.array([o + rng.normal(0, 3, 2500) * max(1.0, abs(o) / 256) for o in offsets]),
                     dtype=torch.float64, device="cuda").to(getattr(torch, DT[dtype]))
    t[1, 100:] = -top
    t[7, 50:] = -INF
    _check_top(t, 16, temperature)


def _case(n, v, k, dtype, seed, stride=0, rest=False, temperature=1.0, ragged=False):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    teacher = torch.randn(n, v, device="cuda", generator=g) * 3
    noise = torch.randn(n, v, device="cuda", generator=g)
    s = _logits(n, v, dtype, seed, stride)
    s.copy_(teacher + noise)
    val, idx, lse = kq.kq_top_logits(teacher, k, temperature)
    w = torch.rand(n, device="cuda", generator=g) + 0.5
    if ragged:
        length = torch.randint(0, k + 1, (n, 1), device="cuda", generator=g)
        idx = torch.where(torch.arange(k, device="cuda") < length, idx, -1).to(torch.int32)
        w[::3] = 0.0
    return s, val, idx, (lse if rest else None), temperature, w


def _bounds(s, val, idx, lse, temperature, w):
    """(loss, gradient) of the oracle and how far from them the GPU may be."""
    sn, vn, ixn = _np(s), host(val), host(idx)
    ln, wn = None if lse is None else host(lse), host(w).astype(np.float64)
    loss, grad, stats = head.distill(sn, vn, ixn, ln, temperature, wn)
    z = np.max(np.where(np.isfinite(sn), np.abs(sn), 0.0), 1) / temperature
    ltol = wn * temperature ** 2 * (1e-4 + 2.0 ** -21 * z)
    # q (P + r / q_r) + p, from the oracle's parts: |gradient| alone may cancel
    n, v = sn.shape
    with np.errstate(all="ignore"):
        q = np.nan_to_num(np.exp((sn.astype(np.float64) - stats[:, :1]) / temperature - stats[:, 1:2]))
        ratio = np.nan_to_num(np.exp(-stats[:, 2]), posinf=0.0)
    p = np.zeros((n, v))
    for i in range(n):
        for j, t in zip(ixn[i], vn[i]):
            if 0 <= j < v:
                zt = ln[i] if ln is not None else max(
                    (vn[i][m] / temperature for m in range(len(ixn[i])) if 0 <= ixn[i][m] < v))
                p[i, j] += np.exp(t / temperature - zt)
    rfac = 1.0 + (ratio[:, None] if lse is not None else 0.0)
    gtol = (wn * temperature)[:, None] * 1e-4 * (q * rfac + np.minimum(p, 2.0))
    return loss, grad, ltol, gtol


def _close(got, want, tol, dtype="f32"):
    got = got.astype(np.float64)
    lo, hi = want - tol - 1e-38, want + tol + 1e-38
    if dtype == "bf16":
        lo, hi = bf16(lo), bf16(hi)
    with np.errstate(invalid="ignore"):
        bad = ~(((lo <= got) & (got <= hi)) | (got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (int(bad.sum()), got[bad][:5], want[bad][:5], np.broadcast_to(tol, got.shape)[bad][:5])


def _check_distill(dtype, s, val, idx, lse, temperature, w):
    loss, grad, ltol, gtol = _bounds(s, val, idx, lse, temperature, w)
    kw = dict(t_lse=lse, temperature=temperature)
    got, stats = kq.kq_distill_loss(s, val, idx, weight=w, **kw)
    _close(host(got), loss, ltol)
    l2, g2 = kq.kq_distill_loss_grad(s, val, idx, weight=w, **kw)
    _close(host(l2), loss, ltol)
    _close(_np(g2), grad, gtol, dtype)
    g3 = kq.kq_distill_grad(s, val, idx, stats, w, **kw)
    _close(_np(g3), grad, gtol, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("n,v,k,stride,t,ragged", [
    (1, 1, 1, 0, 1.0, False), (4, 3, 2, 0, 2.0, True), (6, 100, 30, 5, 1.0, True), (3, 256, 256, 0, 1.0, False),
    (7, 1001, 17, 2, 0.7, True), (2, 32000, 64, 0, 2.0, False), (3, 50001, 100, 47, 1.0, True),
    (2, 128256, 128, 0, 2.0, False), (1, 164001, 200, 0, 1.0, False), (600, 515, 4, 0, 1.0, True),
    (1, 524288, 256, 3, 2.0, False), (270, 16385, 20, 1, 1.0, True)])
def test_distill(n, v, k, stride, t, ragged, rest, dtype):
    print(f"[distill] {n} x {v} k {k} {dtype} rest {rest}", flush=True)
    _check_distill(dtype, *_case(n, v, k, dtype, n + v, stride, rest, t, ragged))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rest", [False, True])
def test_distill_masked_columns_and_odd_lists(rest, dtype):
    s, val, idx, lse, t, w = _case(10, 700, 12, dtype, 8, 0, rest)
    s = s.contiguous()
    low = torch.finfo(s.dtype).min
    s[0, 200:] = -INF             # masked vocabulary; the list may point into it
    s[1, 200:] = low
    s[2, :] = -INF                # no logit at all
    s[3, :] = low                 # every logit the lowest value: uniform
    idx[4, :] = -1                # no list
    idx[5, 3:] = 700              # entries past the vocabulary are none
    idx[5, 2] = 2 ** 31 - 1
    idx[6, 5] = idx[6, 4]         # a column twice
    idx[6, 6] = idx[6, 4]
    val[7, 4:] = -INF             # entries without mass
    s[8, :] = float("nan")
    w[8] = 0.0                    # what has no weight is not looked at
    s[9, 650] = float("nan")
    _check_distill(dtype, s, val, idx, lse, t, w)


def test_distill_list_covers_the_vocabulary():
    """Nothing is off the list: no mass is left for the bucket."""
    for dtype in ("f32", "bf16"):
        _check_distill(dtype, *_case(5, 48, 48, dtype, 3, 0, True, 1.0))


def test_distill_remainder_at_its_limit():
    """A teacher's remainder at most 2^-16 counts as none, one just above it
    counts (t_values are logarithms of the masses, t_lse is 0)."""
    s = _logits(2, 50, "f32", 1)
    p = torch.tensor([[1 - 2.0 ** -17, 0.0], [1 - 2.0 ** -14, 0.0]], device="cuda")
    val = torch.log(p)
    idx = torch.tensor([[3, 9], [3, 9]], dtype=torch.int32, device="cuda")
    lse = torch.zeros(2, device="cuda")
    _check_distill("f32", s, val, idx, lse, 1.0, torch.ones(2, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(5, 3001), (300, 9000), (3, 170001)])
def test_distill_in_place_strides_and_streams(n, v, dtype):
    s, val, idx, lse, t, w = _case(n, v, 9, dtype, 2, 6, True, 2.0, True)
    kw = dict(t_lse=lse, temperature=t)
    loss, grad = kq.kq_distill_loss_grad(s, val, idx, weight=w, **kw)
    _, stats = kq.kq_distill_loss(s, val, idx, weight=w, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    l2, g2 = kq.kq_distill_loss_grad(s, val, idx, weight=w, stream=side, **kw)
    side.synchronize()
    assert torch.equal(loss, l2) and torch.equal(grad, g2)
    buf = torch.full((n, v + 3), 5.0, dtype=s.dtype, device="cuda")
    kq.kq_distill_loss_grad(s, val, idx, weight=w, grad=buf[:, 1:v + 1], **kw)
    assert torch.equal(buf[:, 1:v + 1], grad)
    assert (buf[:, 0] == 5).all() and (buf[:, v + 1:] == 5).all()
    a = s.clone(memory_format=torch.contiguous_format)
    g3 = kq.kq_distill_grad(a, val, idx, stats, w, grad=a, **kw)
    assert g3 is a and torch.equal(a, kq.kq_distill_grad(s, val, idx, stats, w, **kw))
    _, g4 = kq.kq_distill_loss_grad(s, val, idx, weight=w, grad=s, **kw)
    assert torch.equal(g4, grad)


def test_gradient_against_differences_of_the_gpu_losses():
    """Central differences in 16 directions: h = 0.05 leaves h^2 / 6 of a third
    derivative below 1, and 2e-5 of loss error over 2 h."""
    n, v, k = 4, 900, 20
    s, val, idx, lse, t, _ = _case(n, v, k, "f32", 6, 0, True, 1.0)
    _, grad = kq.kq_distill_loss_grad(s, val, idx, t_lse=lse)
    g = torch.Generator(device="cuda").manual_seed(9)
    h = 0.05
    for _ in range(16):
        u = torch.randn(n, v, device="cuda", generator=g)
        up, _ = kq.kq_distill_loss(s + h * u, val, idx, t_lse=lse)
        dn, _ = kq.kq_distill_loss(s - h * u, val, idx, t_lse=lse)
        want = (grad.double() * u.double()).sum(1)
        err = ((up.double() - dn.double()) / (2 * h) - want).abs().max().item()
        assert err < 4 * h * h + 2e-5 / h, err


def test_rest_of_a_list_of_nearly_all_the_mass():
    """A sure teacher at a temperature, t / T near 80 where fp32 steps are
    7.6e-6: t / T of the list rounds as in the log-sum-exp that the caller
    took, so the rest (5e-5 to 1e-3) is what these two leave. Bound of the
    listed column's gradient T (q P - p), of terms near 1: an exponential (2^-23)
    and four roundings on either side of the difference, 1e-6."""
    n, v, T = 64, 1000, 0.7
    rng = np.random.default_rng(8)
    others = rng.normal(0, 3, (n, v)) + rng.uniform(30, 40, (n, 1))
    rest = np.geomspace(5e-5, 1e-3, n)
    others[:, 5] = -1e9
    sure = T * (np.log(np.exp(others / T - 50).sum(1)) + 50 - np.log(rest))
    others[:, 5] = sure
    teacher = torch.tensor(others, dtype=torch.float32, device="cuda")
    student = teacher + torch.tensor(rng.normal(0, 0.3, (n, v)), dtype=torch.float32, device="cuda")
    scaled = teacher * (torch.ones((), device="cuda") / T)
    lse = torch.logsumexp(scaled, 1)
    idx = torch.full((n, 1), 5, dtype=torch.int32, device="cuda")
    val = teacher[:, 5:6].contiguous()
    _, grad = kq.kq_distill_loss_grad(student, val, idx, t_lse=lse, temperature=T)
    T64 = float(np.float32(T))
    as_rounded = host(scaled[:, 5:6]).astype(np.float64) * T64
    _, want, _ = head.distill(host(student), as_rounded, host(idx), host(lse), T64, None)
    assert np.abs(want[:, 5]).max() > 1e-5
    err = np.abs(host(grad)[:, 5] - want[:, 5]).max()
    assert err <= 1e-6, err


def test_no_rows_and_graph_replays():
    e = torch.empty(0, 50, device="cuda")
    v, i, lse = kq.kq_top_logits(e, 4)
    assert v.shape == (0, 4) and lse.shape == (0,)
    loss, grad = kq.kq_distill_loss_grad(e, v, i)
    assert loss.shape == (0,) and grad.shape == (0, 50)
    s, val, idx, lse, t, w = _case(6, 5000, 10, "bf16", 1, 0, True)
    static = s.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        top = kq.kq_top_logits(static, 30)
        out = kq.kq_distill_loss_grad(static, val, idx, t_lse=lse, weight=w)
    for rep in range(3):
        static.copy_(s * (rep + 1))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(top + out, kq.kq_top_logits(static, 30) +
                        kq.kq_distill_loss_grad(static, val, idx, t_lse=lse, weight=w)):
            assert torch.equal(a, b), rep


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows of a 4.4 GB matrix."""
    n, v = 17000, 128256
    s = torch.zeros(n, v, dtype=torch.bfloat16, device="cuda")
    tail = _logits(3, v, "bf16", 12)
    s[-3:] = tail
    val, idx, lse = kq.kq_top_logits(s, 8)
    a, b, c = kq.kq_top_logits(tail, 8)
    assert torch.equal(val[-3:], a) and torch.equal(idx[-3:], b) and torch.equal(lse[-3:], c)
    assert torch.equal(idx[0].cpu(), torch.arange(8, dtype=torch.int32))
    kw = dict(t_lse=c, weight=torch.ones(3, device="cuda"))
    want = kq.kq_distill_loss_grad(tail, a, b.flip(0).contiguous(), **kw)
    w = torch.zeros(n, device="cuda")
    w[-3:] = 1
    idx[-3:] = idx[-3:].flip(0)
    got = kq.kq_distill_loss_grad(s, val, idx, t_lse=lse, weight=w, grad=s)
    assert torch.equal(got[0][-3:], want[0]) and torch.equal(got[1][-3:], want[1])
    assert not got[0][:-3].any() and not got[1][:5].any()

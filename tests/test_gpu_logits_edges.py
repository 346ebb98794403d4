"""GPU tests of the top logits and the distillation loss where rows are out of
the ordinary: equal logits, infinities, mass far below the largest logit,
masks of any value, lists that hold nearly all of the teacher's mass.

Bounds are those of tests/test_gpu_logits.py unless a test derives its own.
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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(3000, 700), (2000, 9000), (1100, 31000), (600, 40000), (300, 60001), (300, 140001)])
def test_top_logits_of_rows_whose_groups_agree(n, v, dtype):
    """Rows of one value, and rows whose largest few are equal in every part of
    the row: the threshold is known without a search. Many rows, so that a
    workgroup goes from one to the next."""
    dt = getattr(torch, DT[dtype])
    c = torch.arange(n, device="cuda").remainder(7).float() - 3.0
    flat = c[:, None].expand(n, v).to(dt).contiguous()
    for k in (1, 5, 64):
        values, index, lse = kq.kq_top_logits(flat, k)
        assert torch.equal(values, c[:, None].expand(n, k))
        assert torch.equal(index, torch.arange(k, dtype=torch.int32, device="cuda").expand(n, k))
        want = c.double() + np.log(v)
        assert ((lse.double() - want).abs() <= 4e-5 + 2.0 ** -22 * want.abs()).all()
    flat[:, ::3] -= 1.0
    values, index, lse = kq.kq_top_logits(flat, 5)
    at = torch.tensor([1, 2, 4, 5, 7], dtype=torch.int32, device="cuda")
    assert torch.equal(values, c[:, None].expand(n, 5)) and torch.equal(index, at.expand(n, 5))
    lower = -(-v // 3)
    want = c.double() + np.log(v - lower + lower * np.exp(-1.0))
    assert ((lse.double() - want).abs() <= 4e-5 + 2.0 ** -22 * want.abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [11, 900, 40000, 140000])
def test_log_sum_exp_of_rows_with_infinities(v, dtype):
    """+inf where a logit is +inf, NaN where one is NaN, -inf where none is
    above it; the lists as ever."""
    rng = np.random.default_rng(v)
    z = rng.normal(0, 2, (7, v))
    z[0, v - 1] = INF
    z[1, 3], z[1, v // 2] = INF, INF
    z[2, 2], z[2, v - 2] = INF, np.nan
    z[3, 1] = np.nan
    z[4, :] = -INF
    z[5, :v - 2], z[5, v - 2] = -INF, INF
    t = torch.tensor(z, dtype=torch.float32, device="cuda").to(getattr(torch, DT[dtype]))
    for temperature in (1.0, 0.3):
        values, index, lse = kq.kq_top_logits(t, 9, temperature)
        wv, wi, wl = head.top_logits(_np(t), 9, temperature)
        np.testing.assert_array_equal(host(index), wi)
        np.testing.assert_array_equal(host(values), wv.astype(np.float32))
        got = host(lse)
        assert got[0] == INF and got[1] == INF and got[5] == INF and got[4] == -INF
        assert np.isnan(got[2]) and np.isnan(got[3])
        assert abs(got[6] - wl[6]) <= 4e-5 + 2.0 ** -22 * abs(wl[6])

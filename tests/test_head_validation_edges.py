"""Further argument checks of the top logits, the distillation loss and the 8-bit
product (CPU): rejected on the host, before any launch."""
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

A, B, C = 0x100000, 0x200000, 0x300000


@pytest.mark.parametrize("t", [1e-45, 2.0 ** -127, 1.17e-38, -1.0])
def test_temperatures_without_a_finite_reciprocal(t):
    """1 / T, and log2(e) / T, have to be numbers: NaN came out for T below
    4.3e-39. Subnormal temperatures are refused."""
    calls = [
        lambda: N.lib.kq_top_logits(A, N.KQ_F32, 4, 100, 100, 5, t, B, C, None, None),
        lambda: N.lib.kq_distill_loss(A, N.KQ_F32, 4, 100, 100, B, C, None, 5, t, None, B, None, None),
        lambda: N.lib.kq_distill_grad(A, N.KQ_F32, 4, 100, 100, B, C, None, 5, t, B, B, C, 100, None),
        lambda: N.lib.kq_distill_loss_grad(A, N.KQ_F32, 4, 100, 100, B, C, None, 5, t, None, B, None, C, 100, None),
    ]
    for call in calls:
        assert call() == N.KQ_ERR_ARG
        assert "temperature" in N.lib.kq_last_error().decode()


def test_the_smallest_temperature_is_taken():
    """(no rows: nothing is launched)"""
    assert N.lib.kq_top_logits(None, N.KQ_F32, 0, 100, 100, 5, 2.0 ** -126, None, None, None, None) == N.KQ_OK


def test_output_types_the_product_does_not_write():
    import torch

    from post_weight_quantization_amd import api

    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    w = z(3, 128, dt=torch.int8)
    for dtype in (torch.float16, torch.float64, torch.int8):
        with pytest.raises(ValueError, match="^dtype: expected"):
            api.kq_linear_i8(z(4, 8), w, z(3), dtype=dtype)
        with pytest.raises(ValueError, match="^dtype: expected"):
            api.kq_matmul_i8(z(4, 128, dt=torch.int8), z(4), w, z(3), 8, dtype=dtype)
    # a matrix of the caller's decides for itself
    with pytest.raises(ValueError, match="GPU"):
        api.kq_linear_i8(z(4, 8), w, z(3), y=z(4, 3), dtype=torch.float16)


@pytest.mark.parametrize("n,d,m,within", [
    (1, 4096, 4096, True), (1, 4096, 12288, True), (1, 4096, 12289, False), (1, 2048, 12288, False),
    (1, 16384, 6144, True), (1, 16384, 7168, False), (1, 16385, 4096, False), (2, 4096, 12288, True),
    (2, 8192, 8192, False), (4, 4096, 4096, True), (4, 4096, 5120, False), (3, 4096, 8192, True),
    (8, 2048, 4096, True), (8, 2048, 8192, False), (8, 1024, 8192, True), (8, 1024, 12288, False),
    (9, 512, 512, False)])
def test_which_sizes_round_their_tokens_within_the_product(n, d, m, within):
    """Those need no workspace; where two launches are faster there is one for the
    codes (8 tokens, 2048 -> 12288: 18.3 us within, 11.4 apart)."""
    import ctypes

    b = ctypes.c_size_t()
    assert N.lib.kq_workspace_size(N.KQ_OP_LINEAR_I8, m, d, n, 0, None, ctypes.byref(b)) == N.KQ_OK
    assert (b.value == 0) == within, b.value

"""CPU checks of the sizes the norm's entry points refuse: the kernels index a row with 32-bit integers, so rows and
row counts above 2^30 are turned away on the host (their tensors would fit the device)."""
import pytest

from bit_mixture_experts_top_b200 import e4b

B = 1 << 40          # tensors far apart


def _norm(T, H, q_format=0):
    q = (6 * B, 7 * B) if q_format else (None, None)
    return e4b.lib().e4b_rmsnorm(B, 2 * B, 3 * B, T, H, 1e-6, q_format, 4 * B, 5 * B, *q, None, None)


def _backward(T, H):
    return e4b.lib().e4b_rmsnorm_backward(B, 0, 2 * B, 3 * B, 4 * B, 5 * B, T, H, 6 * B, 7 * B, 8 * B, B, None)


@pytest.mark.parametrize("T,H", [(1, 2 ** 31 - 1), (1, 2 ** 31 - 64), (1, 2 ** 30 + 1), (2 ** 31 - 1, 8), (2 ** 30 + 1, 1)])
def test_sizes_above_2_to_the_30_are_refused(T, H):
    assert _norm(T, H) == e4b.E4B_ERR_UNSUPPORTED
    assert _norm(T, H, e4b.E4B_Q8_ROW) == e4b.E4B_ERR_UNSUPPORTED
    assert _backward(T, H) == e4b.E4B_ERR_UNSUPPORTED
    assert e4b.e4b_rmsnorm_backward_workspace_bytes(T, H) == 0
    assert _norm(0, H) == (e4b.E4B_OK if H <= 2 ** 30 else e4b.E4B_ERR_UNSUPPORTED)

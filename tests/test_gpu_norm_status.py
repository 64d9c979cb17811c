"""The norm backward's workspace holds the device status word after every call, that of no rows among them."""
import pytest
import torch

from bit_mixture_experts_top_b200 import e4b
from helpers import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [0, 3])
def test_status_word_is_written_by_every_call(T):
    H = 64
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=device())  # noqa: E731
    ws = torch.full((e4b.e4b_rmsnorm_backward_workspace_bytes(T, H),), 7, dtype=torch.uint8, device=device())
    dw = torch.full((H,), 5.0, device=device())
    e4b.e4b_rmsnorm_backward(z(T, H), e4b.E4B_BF16, None, z(T, H), z(H), z(T, dtype=torch.float32), T, H, z(T, H), dw, ws)
    assert e4b.e4b_device_status(ws) == e4b.E4B_OK and not dw.any()


def test_no_rows_need_no_workspace():
    dw = torch.full((64,), 5.0, device=device())
    assert e4b.lib().e4b_rmsnorm_backward(None, 0, None, None, None, None, 0, 64, None, dw.data_ptr(), None, 0,
                                          e4b._stream(None)) == e4b.E4B_OK
    assert not dw.any()

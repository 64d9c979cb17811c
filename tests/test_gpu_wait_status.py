"""A bounded wait that ran out is reported by e4b_wait_status and block.check_waits when its workspace is gone, and on
every device call path that drops its workspace.  (The wait that runs out is the library's own test hook: a barrier
that nothing releases, limited to 2 ms.)"""
import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b
from helpers import device

pytestmark = pytest.mark.gpu


def _run_out(stream=None):
    e4b.e4b_debug_wait_timeout(2_000_000, torch.zeros(4096, dtype=torch.uint8, device=device()), stream)


def test_reported_once_without_the_workspace():
    e4b.e4b_wait_status()                                   # (other tests may have left one)
    assert e4b.e4b_wait_status() == e4b.E4B_OK
    block.check_waits()
    _run_out()
    with pytest.raises(e4b.E4BError, match="TIMEOUT"):
        block.check_waits(device())
    block.check_waits(device())
    _run_out()
    assert e4b.e4b_wait_status() == e4b.E4B_ERR_TIMEOUT and e4b.e4b_wait_status() == e4b.E4B_OK


def test_kept_over_calls_that_clear_their_own_status():
    e4b.e4b_wait_status()
    x = torch.ones((40, 64), dtype=torch.bfloat16, device=device())
    w = torch.ones((256, 64), dtype=torch.bfloat16, device=device())
    ffn, norm = block.GluFfn(w, w[:64, :].repeat(1, 2).contiguous()), block.RmsNorm(x[0].clone())
    side = torch.cuda.Stream()
    ws = torch.zeros(4096, dtype=torch.uint8, device=device())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        e4b.e4b_debug_wait_timeout(2_000_000, ws)
    ffn.forward(x)
    y, r, rstd = norm.forward_train(x)
    norm.backward(y, r, rstd)
    torch.cuda.synchronize()
    assert e4b.e4b_wait_status() == e4b.E4B_ERR_TIMEOUT
    assert e4b.e4b_device_status(ws) == e4b.E4B_ERR_TIMEOUT  # the workspace's own word is another one


def test_calls_that_end_well_report_nothing():
    e4b.e4b_wait_status()
    x = torch.ones((40, 64), dtype=torch.bfloat16, device=device())
    w = torch.ones((256, 64), dtype=torch.bfloat16, device=device())
    ffn = block.GluFfn(w, w[:64, :].repeat(1, 2).contiguous())
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out, saved = ffn.forward_train(x)
        ffn.backward(saved, out)
    g.replay()
    block.check_waits()

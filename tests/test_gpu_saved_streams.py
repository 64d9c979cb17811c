"""A backward on another stream than its forward, its saved state dropped at once: the memory of the saved tensors must
not be handed out again on the forward's stream before the backward has ended.  The backward is held up by a sleep on
its stream; what the forward's stream then allocates and fills would otherwise be what the backward reads."""
import pytest
import torch

from bit_mixture_experts_top_b200 import block
from helpers import device
from test_gpu_block import W, Setup

pytestmark = pytest.mark.gpu


def _refill(sizes):
    """As many allocations of each size as could have been freed, all bits set."""
    return [torch.full((n,), 0xFF, dtype=torch.uint8, device=device()) for n in sizes for _ in range(4)]


def _elsewhere(backward):
    """backward() on a side stream behind a sleep of about 20 ms."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
        got = backward()
    return side, got


@pytest.mark.parametrize("T", [20, 700])
def test_feed_forward(T):
    g = torch.Generator(device=device()).manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device=device()).to(torch.bfloat16)  # noqa: E731
    ffn = block.GluFfn(r(512, 512) / 22, r(512, 256) / 16)
    x, dout = r(T, 512), r(T, 512)
    want = ffn.backward(ffn.forward_train(x)[1], dout)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    saved = [ffn.forward_train(x.clone())[1]]
    sizes = [saved[0].ws.numel(), x.nbytes]
    side, got = _elsewhere(lambda: ffn.backward(saved.pop(), dout))
    junk = _refill(sizes)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    del junk


@pytest.mark.parametrize("name", sorted(W))
def test_block(name):
    s = Setup(W[name], 300)

    def backward(saved):
        return s.block.backward(saved, s.d["dout"], s.d["dr"], router_grad=lambda dl: dl @ s.d["rw"].float())
    train = lambda: s.block.forward_train(s.d["x"], s.d["res"])[2]  # noqa: E731
    want = backward(train())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    saved = [train()]
    sizes = sorted({t.nbytes for t in saved[0] if isinstance(t, torch.Tensor)} | {saved[0][4].ws.nbytes})
    side, got = _elsewhere(lambda: backward(saved.pop()))
    junk = _refill(sizes)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for k in want:
        assert want[k] is None or torch.equal(got[k], want[k]), k
    del junk

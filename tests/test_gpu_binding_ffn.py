"""The feed-forward entry points through the binding, with buffers that the caller owns: the bits of block.GluFfn, with a
workspace larger than asked for and used again, and nothing written beside the outputs."""
import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b
from helpers import device

pytestmark = pytest.mark.gpu
GLU = (1.702, 7.0, 1.0)


@pytest.mark.parametrize("T", [3, 40, 700])
@pytest.mark.parametrize("glu", [None, GLU])
def test_calls_with_the_callers_buffers(T, glu):
    H, I = 264, 136
    g = torch.Generator(device=device()).manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device=device())  # noqa: E731
    bf = lambda *s: rand(*s).to(torch.bfloat16)  # noqa: E731
    gu, dn, x, add, dout = bf(2 * I, H) / 16, bf(H, I) / 12, bf(T, H), bf(T, H), bf(T, H)
    bg, bd = rand(2 * I), rand(H)
    ffn = block.GluFfn(gu, dn, bg, bd, glu)
    desc = e4b.make_ffn_desc(H, I, glu)
    ws = torch.full((e4b.e4b_ffn_train_workspace_bytes(desc, T) + 512,), 7, dtype=torch.uint8, device=device())
    out = torch.full((T + 1, H), 5.0, dtype=torch.bfloat16, device=device())
    e4b.e4b_ffn_forward(desc, T, x, gu, dn, bg, bd, add, out[:T], ws)
    assert torch.equal(out[:T], ffn.forward(x, add)) and e4b.e4b_device_status(ws) == e4b.E4B_OK
    out.fill_(5.0)
    e4b.e4b_ffn_forward_train(desc, T, x, gu, dn, bg, bd, add, out[:T], ws)
    want, saved = ffn.forward_train(x, add)
    assert torch.equal(out[:T], want) and bool((out[T:] == 5).all()) and bool((ws[-512:] == 7).all())
    full = ffn.backward(saved, dout)
    outs = [torch.full_like(t, 3.0) for t in full]
    e4b.e4b_ffn_backward(desc, T, x, dout, gu, dn, *outs, ws)
    for a, b in zip(outs, full):
        assert torch.equal(a, b)
    assert e4b.e4b_device_status(ws) == e4b.E4B_OK and bool((ws[-512:] == 7).all())

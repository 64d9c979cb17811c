"""CPU checks of what block.MoeBlock keeps between its calls, with the entry points of the routed layer replaced by
fakes that write their call's number into the workspace: every call has a workspace of its own, and a backward gets
the one that its own forward filled."""
import contextlib

import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b, layer

E, H, I, K = 8, 256, 128, 2


class FakeNorm:
    """Stands in for block.RmsNorm on the CPU."""
    index = -1

    def __init__(self):
        self.H = H

    def forward(self, x, residual=None):
        return x.clone(), x

    def forward_train(self, x, residual=None):
        return x.clone(), x, torch.ones(len(x))

    def backward(self, dy, r, rstd, dr=None):
        return dy, torch.zeros(H)


@pytest.fixture
def calls(monkeypatch):
    """The list of ("forward" / "train" / "backward", workspace) of every call into the routed layer."""
    made = []

    def forward(kind):
        def call(desc, T, *args):
            ws = args[-2]
            query = e4b.e4b_moe_workspace_bytes if kind == "forward" else e4b.e4b_moe_train_workspace_bytes
            assert ws.numel() >= query(desc, T)
            ws[256:264] = len(made)
            made.append((kind, ws))
        return call

    def backward(desc, T, *args):
        made.append(("backward", args[-2]))
    monkeypatch.setattr(e4b, "e4b_moe_forward", forward("forward"))
    monkeypatch.setattr(e4b, "e4b_moe_forward_train", forward("train"))
    monkeypatch.setattr(e4b, "e4b_moe_backward", backward)
    monkeypatch.setattr(block, "_check", lambda t, *a: t)
    monkeypatch.setattr(block, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(block, "_on", lambda index, *t: contextlib.nullcontext())
    return made


def _block():
    stack = lambda n, k: layer.PackedStack(torch.empty(1), torch.empty(1), E, n, k, "nf4")  # noqa: E731
    moe = layer.MoeLayer(E, H, I, K, "nf4", stack(2 * I, H), stack(H, I))
    return block.MoeBlock(FakeNorm(), lambda y: torch.zeros((len(y), E), dtype=torch.bfloat16), moe)


def _x(T):
    return torch.zeros((T, H), dtype=torch.bfloat16)


def test_each_backward_gets_the_workspace_of_its_own_forward(calls):
    b = _block()
    saved = [b.forward_train(_x(T))[2] for T in (5, 64, 5)]
    for i in (1, 0, 2):
        b.backward(saved[i], _x(len(saved[i][0])))
        assert int(calls[-1][1][256]) == i


def test_an_evaluation_between_forward_and_backward_leaves_the_saved_state(calls):
    b = _block()
    _, _, saved = b.forward_train(_x(40))
    for T in (40, 3, 900):
        b.forward(_x(T))
    b.backward(saved, _x(40))
    assert int(calls[-1][1][256]) == 0


def test_calls_share_no_workspace(calls):
    b = _block()
    for T in (4, 4, 900, 4):
        b.forward(_x(T))
    saved = [b.forward_train(_x(4))[2] for _ in range(2)]
    assert len({ws.data_ptr() for _, ws in calls}) == 6 and len(saved) == 2

"""CPU checks of what block.MoeBlock refuses before the routed layer's entry points get any pointer, with tensors that
only claim to be on a GPU and entry points that fail the test when they are reached."""
import contextlib

import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b, layer
from test_block_state import E, H, I, K, FakeNorm


class Claims(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    is_cuda = True


def _claims(t):
    return t.as_subclass(Claims)


def _x(T):
    return _claims(torch.zeros((T, H), dtype=torch.bfloat16))


@pytest.fixture
def blk(monkeypatch):
    reached = []
    monkeypatch.setattr(e4b, "e4b_moe_forward_train", lambda *a: None)
    monkeypatch.setattr(e4b, "e4b_moe_backward", lambda *a: reached.append(a))
    monkeypatch.setattr(block, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(block, "_on", lambda index, *t: contextlib.nullcontext())
    stack = lambda n, k: layer.PackedStack(torch.empty(1), torch.empty(1), E, n, k, "nf4")  # noqa: E731
    moe = layer.MoeLayer(E, H, I, K, "nf4", stack(2 * I, H), stack(H, I))
    b = block.MoeBlock(FakeNorm(), lambda y: _claims(torch.zeros((len(y), E), dtype=torch.bfloat16)), moe)
    b.reached = reached
    return b


def test_backward_takes_a_contiguous_gradient_of_the_saved_rows(blk):
    _, _, saved = blk.forward_train(_x(6))
    blk.backward(saved, _x(6))
    assert len(blk.reached) == 1
    one = _claims(torch.ones((), dtype=torch.bfloat16))
    for bad in (one.expand(6, H),                            # as a sum's gradient comes: one value, no rows behind it
                _x(6)[:3], _x(7), _claims(torch.zeros((6, H))), _x(6)[:, : H // 2],
                _claims(torch.zeros((H, 6), dtype=torch.bfloat16)).t(), torch.zeros((6, H), dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="dout"):
            blk.backward(saved, bad)
    assert len(blk.reached) == 1


def test_every_call_runs_on_the_device_of_the_block(blk, monkeypatch):
    inside, seen = [], []

    @contextlib.contextmanager
    def on(index, *tensors):
        inside.append((index, [t for t in tensors if t is not None]))
        yield
        inside.pop()
    monkeypatch.setattr(block, "_on", on)
    for name in ("e4b_moe_forward", "e4b_moe_forward_train", "e4b_moe_backward"):
        monkeypatch.setattr(e4b, name, lambda *a, name=name: seen.append((name, len(inside))))
    router, grads = blk.router, lambda dl: seen.append(("router_grad", len(inside))) or torch.zeros((len(dl), H))
    blk.router = lambda y: seen.append(("router", len(inside))) or router(y)
    blk.forward(_x(5))
    _, _, saved = blk.forward_train(_x(5))
    blk.backward(saved, _x(5), router_grad=grads)
    assert [n for n, _ in seen] == ["router", "e4b_moe_forward", "router", "e4b_moe_forward_train", "e4b_moe_backward",
                                    "router_grad"]
    assert all(depth > 0 for _, depth in seen), seen


def test_parts_on_different_devices_are_refused():
    stack = lambda n, k: layer.PackedStack(torch.empty(1), torch.empty(1), E, n, k, "nf4")  # noqa: E731
    moe = layer.MoeLayer(E, H, I, K, "nf4", stack(2 * I, H), stack(H, I))
    elsewhere = FakeNorm()
    elsewhere.index = 1
    with pytest.raises(ValueError, match="device"):
        block.MoeBlock(elsewhere, None, moe)

    class FakeShared:
        H, index = FakeNorm().H, 1
    with pytest.raises(ValueError, match="device"):
        block.MoeBlock(FakeNorm(), None, moe, FakeShared())


def test_saved_state_of_another_layer_is_refused(blk, monkeypatch):
    # its routing and row counts would be read as this layer's
    _, _, saved = blk.forward_train(_x(6))
    stack = lambda e, n, k: layer.PackedStack(torch.empty(1), torch.empty(1), e, n, k, "nf4")  # noqa: E731
    same = layer.MoeLayer(E, H, I, K, "nf4", stack(E, 2 * I, H), stack(E, H, I))
    block.MoeBlock(blk.norm, blk.router, same).backward(saved, _x(6))
    assert len(blk.reached) == 1
    for e, i, k in ((4, I, K), (E, 2 * I, K), (E, I, 1)):
        other = layer.MoeLayer(e, H, i, k, "nf4", stack(e, 2 * i, H), stack(e, H, i))
        with pytest.raises(ValueError, match="saved"):
            block.MoeBlock(blk.norm, blk.router, other).backward(saved, _x(6))
    assert len(blk.reached) == 1


def test_saved_state_of_another_feed_forward_block_is_refused(monkeypatch):
    monkeypatch.setattr(block, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(block, "_on", lambda index, *t: contextlib.nullcontext())
    reached = []
    monkeypatch.setattr(e4b, "e4b_ffn_backward", lambda *a: reached.append(a))
    z = lambda *s: _claims(torch.zeros(s, dtype=torch.bfloat16))  # noqa: E731
    make = lambda h, i, glu=None: block.GluFfn(z(2 * i, h), z(h, i), glu=glu)  # noqa: E731
    ffn = make(64, 128)
    saved = block.FfnSaved(z(5, 64), torch.empty(1), 0, ffn.desc)
    make(64, 128).backward(saved, z(5, 64))
    assert len(reached) == 1
    for other in (make(64, 256), make(128, 128), make(64, 128, (1.702, 7.0, 1.0))):
        with pytest.raises(ValueError, match="saved"):
            other.backward(saved, z(5, other.H))
    assert len(reached) == 1

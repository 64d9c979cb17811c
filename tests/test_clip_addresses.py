"""CPU checks that block.GradClipper hands the library the addresses its tensors have now, with the library replaced by
a fake that reads the table: a tensor may be given other storage between two calls."""
import contextlib
import ctypes

import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b


class FakeLibrary:
    """Keeps the table of the last call as (grad, out, n, dtype) tuples."""

    def e4b_clip_grad_norm_workspace_bytes(self, n):
        return 256

    def e4b_clip_grad_norm(self, table, n, *rest):
        a = (e4b.Grad * n).from_address(table)
        self.table = [(g.grad, g.out, g.n, g.dtype) for g in a]
        return e4b.E4B_OK


@pytest.fixture
def lib(monkeypatch):
    fake = FakeLibrary()
    monkeypatch.setattr(e4b, "lib", lambda: fake)
    monkeypatch.setattr(e4b, "_need_cuda", lambda *t: None)
    monkeypatch.setattr(e4b, "_stream", lambda s: None)
    monkeypatch.setattr(block, "_on", lambda index, *t: contextlib.nullcontext())
    return fake


def _now(grads, outs):
    return [(g.data_ptr(), o.data_ptr(), g.numel(), e4b.DTYPES[g.dtype]) for g, o in zip(grads, outs)]


@pytest.mark.parametrize("in_place", [True, False])
def test_tensors_given_other_storage_are_followed(lib, in_place):
    grads = [torch.ones(n) for n in (5, 70, 3)]
    outs = grads if in_place else [torch.ones(n) for n in (5, 70, 3)]
    c = block.GradClipper(grads, None if in_place else outs)
    c.clip(1.0)
    assert lib.table == _now(grads, outs)
    for change in (lambda t: setattr(t, "data", torch.ones(t.numel())), lambda t: t.set_(torch.ones(t.numel())),
                   lambda t: setattr(t, "data", torch.ones(t.numel() + 7)), lambda t: t.resize_(100000)):
        for t in {id(t): t for t in grads + outs}.values():
            change(t)
            if not in_place:                      # a pair has one size
                for g, o in zip(grads, outs):
                    if g.numel() != o.numel():
                        (o if t is g else g).data = torch.ones(t.numel())
            c.clip(1.0)
            assert lib.table == _now(grads, outs)


def test_storage_that_the_table_names_is_not_freed_before_the_next_call(lib):
    import weakref
    t = torch.ones(1000)
    c = block.GradClipper([t])
    old = weakref.ref(t.untyped_storage())
    t.data = torch.ones(1000)
    assert old() is not None                      # so nothing else can come to lie at the address in the table
    c.clip(1.0)
    assert old() is None and lib.table == _now([t], [t])


def test_a_change_that_cannot_be_described_is_refused(lib):
    t = torch.ones(8, 8)
    c = block.GradClipper([t])
    t.data = torch.ones(8, 8).t()
    for _ in range(2):
        with pytest.raises(ValueError, match="contiguous"):
            c.clip(1.0)
    t.data = torch.ones(8, 8, dtype=torch.float64)
    with pytest.raises(ValueError):
        c.clip(1.0)
    t.data = torch.ones(8, 8, dtype=torch.float16)
    c.clip(1.0)
    assert lib.table == _now([t], [t]) and ctypes.sizeof(c.grads) == ctypes.sizeof(e4b.Grad)

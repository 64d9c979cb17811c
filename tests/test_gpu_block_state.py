"""block.MoeBlock called in every order that its documentation allows: other calls between a training forward and its
backward, two graphs of one block at once, and a replay after a call with more tokens.  The kernels give the same
bits for the same inputs, so every comparison is exact."""
import pytest
import torch

from test_gpu_block import W, Setup, _step

pytestmark = pytest.mark.gpu
NAMES = sorted(W)


def _train(s):
    return s.block.forward_train(s.d["x"], s.d["res"])


def _back(s, saved):
    return s.block.backward(saved, s.d["dout"], s.d["dr"], router_grad=lambda dl: dl @ s.d["rw"].float())


def _same(a, b):
    for k in a:
        assert (a[k] is None and b[k] is None) or torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("name", NAMES)
def test_backwards_after_other_calls(name):
    a, b = Setup(W[name], 40), Setup(W[name], 300)
    b.block = a.block
    want = [_step(s)[2] for s in (a, b)]
    sa, sb = _train(a)[2], _train(b)[2]
    for s in (b, a):                             # evaluations with more and with fewer tokens
        s.block.forward(s.d["x"], s.d["res"])
    _same(_back(a, sa), want[0])
    _same(_back(b, sb), want[1])
    _same(_back(a, sa), want[0])                 # the saved state survives its backward


@pytest.mark.parametrize("name", NAMES)
def test_two_graphs_of_one_block_and_a_larger_call_between(name):
    a, b = Setup(W[name], 40), Setup(W[name], 64)
    b.block = a.block
    want = [_step(s) for s in (a, b)]
    graphs, got = [], []
    torch.cuda.synchronize()
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(_step(s))
        graphs.append(g)
    big = Setup(W[name], 900)
    big.block = a.block
    big.block.forward(big.d["x"], big.d["res"])  # more tokens than either graph was captured with
    _step(big)
    fill = [torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(64)]
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
        _same(x[2], y[2])
    assert all(bool((t == 0x7F).all()) for t in fill)     # a replay writes nowhere else


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(name):
    a, b = Setup(W[name], 64), Setup(W[name], 300)
    b.block = a.block
    want = [s.block.forward(s.d["x"], s.d["res"])[0] for s in (a, b)]
    streams = [torch.cuda.Stream() for _ in want]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(s.block.forward(s.d["x"], s.d["res"])[0])
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(o, w) for o in outs)


@pytest.mark.parametrize("name", NAMES)
def test_no_tokens(name):
    s = Setup(W[name], 4)
    x = s.d["x"][:0]
    out, r = s.block.forward(x, x)
    assert out.shape == r.shape == x.shape
    out, r, saved = s.block.forward_train(x, x)
    got = s.block.backward(saved, x, x, router_grad=lambda dl: dl @ s.d["rw"].float())
    assert got["dx"].shape == x.shape and got["dlogits"].shape == (0, s.w.E)
    for k in ("norm", "gate_up", "down", "lora_A", "lora_B"):
        assert got[k] is None or not got[k].any(), k

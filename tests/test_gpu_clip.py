"""GPU parity of the gradient norm and clipping (block.GradClipper, e4b_clip_grad_norm) against fp64.

Squares and sums are fp64 (n <= 2^27 terms: below 2^-26 relative), so the norm is one fp32 rounding, 2^-24, off.
The factor is one fp32 rounding of the fp64 quotient and each output one more of its type: at most
2^-24 + 2^-25 + eps / 2, or half the smallest subnormal."""
import numpy as np
import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b
from helpers import device
from oracle import dense

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _grads(sizes, seed=0, types=TYPES, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std * (1 + i % 3)).to(types[i % len(types)]).to(device())
            for i, n in enumerate(sizes)]


def _check(grads, outs, norm, max_norm):
    want, ref = dense.clip_grads([g.double().cpu().numpy() for g in grads], max_norm)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    for g, o, r in zip(grads, outs, ref):
        e = torch.finfo(g.dtype)
        got = o.double().cpu().numpy()
        bound = np.abs(r) * (e.eps / 2 + 2.0 ** -23) + e.smallest_normal * e.eps / 2
        assert (np.abs(got - r) <= bound).all()


SIZES = [[1], [3], [4096], [4097, 1, 0, 2], [0, 0], [0, 5, 0], list(range(1, 40)), [100003, 17, 8192, 70000],
         [3000 + 7 * i for i in range(64)], [11 * i for i in range(65)], [257] * 257, [5] * 961, [13, 70000] * 1000]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{sum(s)}")
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_out_of_place_and_in_place(sizes, max_norm):
    grads = _grads(sizes)
    kept = [g.clone() for g in grads]
    outs = [torch.full_like(g, 7) for g in grads]
    norm = block.GradClipper(grads, outs).clip(max_norm)
    assert norm.shape == () and norm.dtype == torch.float32
    for g, k in zip(grads, kept):
        assert torch.equal(g, k)
    _check(kept, outs, norm, max_norm)
    again = block.GradClipper(grads).clip(max_norm)
    assert torch.equal(again, norm)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)


@pytest.mark.parametrize("types", [[torch.float32], [torch.bfloat16], [torch.float16], TYPES])
def test_packed_without_alignment(types):
    sizes = [1, 2, 3, 5, 1000, 7, 16384 + 3, 9, 33, 50001]
    src = {t: torch.randn(sum(sizes) + 8, generator=torch.Generator().manual_seed(3)).to(t).to(device()) for t in types}
    for gap in (0, 1):                       # outs with the same offsets as the gradients, and with others
        dst = {t: torch.full_like(v, 9) for t, v in src.items()}
        at, grads, outs = 0, [], []
        for i, n in enumerate(sizes):
            t = types[i % len(types)]
            grads.append(src[t][at:at + n])
            outs.append(dst[t][at + gap:at + gap + n])
            at += n
        norm = block.GradClipper(grads, outs).clip(0.25)
        _check(grads, outs, norm, 0.25)
        used = {t: torch.zeros(v.numel(), dtype=torch.bool) for t, v in dst.items()}
        at = 0
        for i, n in enumerate(sizes):
            used[types[i % len(types)]][at + gap:at + gap + n] = True
            at += n
        for t in types:                      # nothing beside the outs is written
            assert bool((dst[t].cpu()[~used[t]] == 9).all())


def test_long_lists():
    # over 160 MB the blocks stride over the list; whole and ragged tensors, all types, unaligned ones among them
    sizes = [25_000_003, 1, 17_000_001, 33, 0, 1 << 20, 12_345_679]
    flat = {t: (torch.randn(30_000_000, generator=torch.Generator(device="cuda").manual_seed(5), device=device())).to(t) for t in TYPES}
    grads, at = [], {t: i for i, t in enumerate(TYPES)}
    for i, n in enumerate(sizes):
        t = TYPES[0] if i in (0, 2) else TYPES[i % 3]
        start = 0 if n > 30_000_000 - at[t] - n else at[t]
        grads.append((torch.randn(n + 1, generator=torch.Generator(device="cuda").manual_seed(i), device=device()).to(t))[1:]
                     if start == 0 else flat[t][start:start + n])
        at[t] = start + n
    outs = [torch.full_like(g, 7) for g in grads]
    assert sum(g.nbytes for g in grads) > 160 << 20
    norm = block.GradClipper(grads, outs).clip(3.0)
    _check(grads, outs, norm, 3.0)
    kept = [g.clone() for g in grads]
    assert torch.equal(block.GradClipper(kept).clip(3.0), norm)
    for k, o in zip(kept, outs):
        assert torch.equal(k, o)


def test_extreme_values():
    big = [torch.full((1000,), 1e30, device=device()), torch.full((10,), 1e-30, device=device())]
    outs = [torch.empty_like(g) for g in big]
    _check(big, outs, block.GradClipper(big, outs).clip(1.0), 1.0)
    tiny = [torch.full((1 << 16,), 1e-30, device=device())]
    norm = block.GradClipper(tiny).clip(1.0)
    assert abs(float(norm) - 256e-30) <= 2.0 ** -22 * 256e-30
    zero = [torch.zeros(100, device=device())]
    assert float(block.GradClipper(zero).clip(1.0)) == 0 and not zero[0].any()
    g = _grads([100, 100], types=[torch.float32])
    outs = [torch.empty_like(t) for t in g]
    assert float(block.GradClipper(g, outs).clip(0.0)) > 0 and not any(bool(o.any()) for o in outs)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite(bad):
    g = _grads([1000, 3, 70000])
    g[2][69999] = bad
    params = [torch.nn.Parameter(torch.zeros_like(t, dtype=torch.float32)) for t in g]
    for p, t in zip(params, g):
        p.grad = t.float().clone()
    want = torch.nn.utils.clip_grad_norm_(params, 1.0, foreach=False)
    norm = block.GradClipper(g).clip(1.0)
    assert torch.equal(torch.isnan(norm), torch.isnan(want)) and torch.equal(torch.isinf(norm), torch.isinf(want))
    for t, p in zip(g, params):
        assert torch.equal(torch.isnan(t), torch.isnan(p.grad))
        assert not torch.nan_to_num(t.float()).any() and not torch.nan_to_num(p.grad).any()
    # the norm alone leaves the values
    h = _grads([1000, 3])
    h[0][5] = bad
    k = [t.clone() for t in h]
    block.GradClipper(h).clip(float("inf"))
    for t, s in zip(h, k):
        assert torch.equal(t.view(torch.uint8), s.view(torch.uint8))


def test_norm_alone():
    g = _grads([100, 70000, 3])
    k = [t.clone() for t in g]
    norm = block.GradClipper(g).clip(float("inf"))
    _check(k, g, norm, float("inf"))
    outs = [torch.empty_like(t) for t in g]
    block.GradClipper(g, outs).clip(float("inf"))
    for t, o in zip(g, outs):
        assert torch.equal(t, o)


def test_no_tensors_through_the_c_entry():
    norm = torch.full((1,), 5.0, device=device())
    ws = torch.empty(e4b.e4b_clip_grad_norm_workspace_bytes(0), dtype=torch.uint8, device=device())
    e4b.e4b_clip_grad_norm(e4b.make_grads([]), 1.0, norm, ws)
    assert float(norm) == 0.0


def test_graph_replay_and_two_clippers_at_once():
    a, b = _grads([70000, 33], 1), _grads([5, 90001], 2)
    oa, ob = [torch.empty_like(t) for t in a], [torch.empty_like(t) for t in b]
    ca, cb = block.GradClipper(a, oa), block.GradClipper(b, ob)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(ga):
        na = ca.clip(0.5)
    with torch.cuda.graph(gb):
        nb = cb.clip(0.5)
    for t in a + b:
        t.mul_(2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(sa):
            ga.replay()
        with torch.cuda.stream(sb):
            gb.replay()
    torch.cuda.synchronize()
    _check(a, oa, na, 0.5)
    _check(b, ob, nb, 0.5)


def test_a_dropped_clipper_lets_its_tensors_go_at_once():
    import gc
    import weakref
    gc.disable()
    try:
        g = _grads([100, 7])
        c = block.GradClipper(g)
        c.clip(1.0)
        e4b.e4b_clip_grad_norm(c.grads, 1.0, torch.empty(1, device=device()),
                               torch.empty(e4b.e4b_clip_grad_norm_workspace_bytes(2), dtype=torch.uint8, device=device()))
        ref = weakref.ref(g[0])
        del g, c
        assert ref() is None
    finally:
        gc.enable()


def test_refusals():
    g = _grads([100, 100])
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        block.GradClipper([g[0], g[0]]).clip(1.0)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        block.GradClipper(g).clip(-1.0)
    with pytest.raises(ValueError, match="contiguous"):
        block.GradClipper([torch.zeros(8, 8, device=device()).t()])
    with pytest.raises(ValueError):
        block.GradClipper([torch.zeros(8, dtype=torch.float64, device=device())])
    with pytest.raises(ValueError):
        block.GradClipper([g[0]], [g[1]])

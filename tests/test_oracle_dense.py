"""Pins for oracle/dense.py: the norm, its 8-bit outputs, the feed-forward block and clipping against torch's
fp64 forms, brute force and central finite differences, none of which share its derivations."""
import numpy as np
import pytest
import torch

from bit_mixture_experts_top_b200 import synth
from oracle import bf16, dense

GLU = (1.702, 7.0, 1.0)


def test_e4m3_rounding_matches_torch_on_values_midpoints_and_random():
    v = dense.e4m3_values()
    assert v[-1] == 448 and v[1] == 2.0 ** -9 and len(v) == 127
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(500)),
                        np.random.default_rng(0).uniform(0, 448, 4000), 2.0 ** np.random.default_rng(1).uniform(-12, 8, 4000)])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(dense.round_to_e4m3(x.astype(np.float64)), want)
    assert dense.round_to_e4m3(np.array([np.nan]))[0] == 0x7F


def test_rmsnorm_matches_torch_fp64_and_is_homogeneous():
    T, H = 5, 96
    x = synth.normal_bf16((T, H), 1.0, 0, "rn_x")
    res = synth.normal_bf16((T, H), 1.0, 0, "rn_r")
    w = synth.normal_bf16((H,), 1.0, 0, "rn_w")
    r_bits, rstd, y = dense.rmsnorm(x, res, w, 1e-5)
    want_r = (torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).double() +
              torch.from_numpy(res.view(np.int16)).view(torch.bfloat16).double()).to(torch.bfloat16)
    assert np.array_equal(r_bits.view(np.int16), want_r.view(torch.int16).numpy())
    want = torch.nn.functional.rms_norm(want_r.double(), (H,), torch.from_numpy(bf16.bf16_bits_to_f64(w)), 1e-5)
    assert np.allclose(y, want.numpy(), rtol=3 * 2.0 ** -24, atol=0)      # rstd and two products round in fp32
    # a row of equal values norms to the weight's sign; a row of zeros to zero
    one = np.full((1, H), 0x4040, np.uint16)
    _, rs, y1 = dense.rmsnorm(one, None, w, 0.0)
    assert np.allclose(y1[0], bf16.bf16_bits_to_f64(w), rtol=3 * 2.0 ** -24)
    assert not dense.rmsnorm(np.zeros((1, H), np.uint16), None, w, 1e-6)[2].any()


def test_mx_and_row_codes_read_back_within_half_a_step():
    g = np.random.default_rng(3)
    y = (g.standard_normal((6, 128)) * np.exp(g.normal(0, 4, (6, 1)))).astype(np.float32)
    y[2] = 0
    y[3, 5] = np.inf
    v = np.concatenate([dense.e4m3_values(), [np.nan]])
    val = np.concatenate([v, -v])
    for codes, scale in [(dense.quantize_mx(y)[0], np.repeat(2.0 ** (dense.quantize_mx(y)[1].astype(float) - 127), 32, axis=1)),
                         (dense.quantize_rows(y)[0], dense.quantize_rows(y)[1][:, None].astype(float))]:
        got = val[codes] * scale
        fine = np.isfinite(got)
        assert not fine[3].all() and fine[[0, 1, 2, 4, 5]].all()
        y0 = np.where(np.isfinite(y), y, 0.0).astype(np.float64)
        # half a step: 2^-4 relative, or half the subnormal step 2^-9
        bound = np.maximum(np.abs(y0) * 2.0 ** -4, np.broadcast_to(scale, y.shape) * 2.0 ** -10) * (1 + 2.0 ** -22)
        assert (np.abs(got - y0)[fine] <= bound[fine]).all()
    s = dense.quantize_mx(y)[1]
    assert s[2].max() == 0 and s[3, 0] == 255 and s[3, 1] != 255
    # amax = 448 * 2^e keeps exponent e, the next fp32 value takes e + 1
    edge = np.zeros((1, 64), np.float32)
    edge[0, 0], edge[0, 32] = 448 * 8, np.nextafter(np.float32(448 * 8), np.float32(1e9))
    assert dense.quantize_mx(edge)[1].tolist() == [[130, 131]]


def _fd(f, a, idx, eps=1e-6):
    b = a.copy()
    b[idx] += eps
    up = f(b)
    b[idx] -= 2 * eps
    return (up - f(b)) / (2 * eps)


def _entries(name, f, a, grad, n=10):
    scale = np.abs(grad).max()
    for i in np.random.default_rng(1).choice(a.size, size=min(n, a.size), replace=False):
        idx = np.unravel_index(i, a.shape)
        assert abs(_fd(f, a, idx) - grad[idx]) <= 2e-6 * scale, (name, idx)


def test_rmsnorm_backward_against_finite_differences():
    g = np.random.default_rng(5)
    T, H, eps = 4, 24, 1e-3
    r, w, dy, dr = g.standard_normal((T, H)), g.standard_normal(H), g.standard_normal((T, H)), g.standard_normal((T, H))

    def loss(r, w):
        return np.sum(dy * r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps) * w) + np.sum(dr * r)
    rstd = 1 / np.sqrt(np.mean(r * r, axis=1) + eps)
    dx, dw = dense.rmsnorm_backward(dy, r, w, rstd, dr)
    _entries("dx", lambda a: loss(a, w), r, dx)
    _entries("dw", lambda a: loss(r, a), w, dw)
    # the gradient does not depend on dy along the row itself up to eps: with eps = 0 dx is orthogonal to r
    rstd0 = 1 / np.sqrt(np.mean(r * r, axis=1))
    assert np.abs(np.sum(dense.rmsnorm_backward(dy, r, w, rstd0)[0] * r, axis=1)).max() < 1e-12


@pytest.mark.parametrize("glu", [None, GLU])
def test_ffn_backward_against_finite_differences(glu):
    g = np.random.default_rng(7)
    T, H, I = 5, 12, 9
    x, wgu, wdn = g.standard_normal((T, H)), g.standard_normal((2 * I, H)), g.standard_normal((H, I))
    bgu, bdn, dout = g.standard_normal(2 * I), g.standard_normal(H), g.standard_normal((T, H))
    if glu:
        wgu *= 2.5            # some gates and ups beyond the clamps

    def loss(x=x, wgu=wgu, wdn=wdn, bgu=bgu, bdn=bdn):
        return float(np.sum(dout * dense.ffn(x, wgu, wdn, bgu, bdn, glu=glu)[0]))
    if glu:
        G = dense.ffn(x, wgu, wdn, bgu, glu=glu)[2]
        assert (G[:, :I] > 7).any() and (np.abs(G[:, I:]) > 7).any() and np.abs(np.abs(G) - 7).min() > 1e-4
    dx, dgu, ddn, dbg, dbd = dense.ffn_backward(x, wgu, wdn, dout, bgu, glu)
    _entries("x", lambda a: loss(x=a), x, dx)
    _entries("wgu", lambda a: loss(wgu=a), wgu, dgu, 20)
    _entries("wdn", lambda a: loss(wdn=a), wdn, ddn)
    _entries("bgu", lambda a: loss(bgu=a), bgu, dbg, 18)
    _entries("bdn", lambda a: loss(bdn=a), bdn, dbd)


def test_ffn_is_linear_in_the_down_weights_and_adds_the_routed_output():
    g = np.random.default_rng(8)
    x, wgu, wdn, add = (g.standard_normal(s) for s in ((3, 8), (10, 8), (8, 5), (3, 8)))
    a = dense.ffn(x, wgu, wdn)[0]
    assert np.allclose(dense.ffn(x, wgu, 2 * wdn, add=add)[0], 2 * a + add)
    t = torch.from_numpy
    want = (torch.nn.functional.silu(t(x) @ t(wgu[:5]).T) * (t(x) @ t(wgu[5:]).T)) @ t(wdn).T
    assert np.allclose(a, want.numpy())


@pytest.mark.parametrize("max_norm", [0.0, 0.3, 1e9, float("inf")])
def test_clip_matches_torch(max_norm):
    g = np.random.default_rng(9)
    grads = [g.standard_normal(n) for n in (1, 7, 300)]
    ps = [torch.nn.Parameter(torch.zeros(len(a), dtype=torch.float64)) for a in grads]
    for p, a in zip(ps, grads):
        p.grad = torch.from_numpy(a.copy())
    norm, out = dense.clip_grads(grads, max_norm)
    want = torch.nn.utils.clip_grad_norm_(ps, max_norm)
    assert np.isclose(norm, float(want), rtol=1e-12)
    for p, o in zip(ps, out):
        assert np.allclose(p.grad.numpy(), o, rtol=1e-12, atol=0)

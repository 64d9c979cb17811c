"""GPU parity of the gated feed-forward block (block.GluFfn, e4b_ffn_*) against oracle/dense.py in fp64.

Per element, with eacc(K) = (K / 16 + 2) 2^-21 for an fp32 accumulation of K products in steps of 16 (each step may
lose 8 units of 2^-24 of the magnitude it adds to), to first order:
  G   : dG0 = eacc(H) (|x| |Wgu|^T + |b|)
  h   : act'-weighted dG0, 2^-18 |h| for the fast exponential, one bf16 rounding 2^-8 |h|
  out : dh-weighted |Wdn|, eacc(I) |h| |Wdn|^T, one bf16 rounding 2^-8 |out|
and the backward's products alike, with dG rounded once to bf16.  Second derivatives of both activations are below
(|u| + |beta| + 1) 1.2.  Beside that the layer's own bounds on relative Frobenius error hold: 5e-3 for the output,
1e-2 for the gradients."""
import numpy as np
import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b, synth
from helpers import bf16_to_f64, device
from oracle import bf16, dense

pytestmark = pytest.mark.gpu
GLU = (1.702, 7.0, 1.0)
B8 = 2.0 ** -8


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device()).view(torch.bfloat16)


class Case:
    def __init__(self, T, H, I, glu=None, bias=False, add=False, wide=1.0):
        self.T, self.H, self.I, self.glu = T, H, I, glu
        bits = lambda shape, name, std=1.0: synth.normal_bf16(shape, std, 0, f"ffn_{name}_{T}_{H}_{I}")  # noqa: E731
        self.b = dict(x=bits((T, H), "x"), gu=bits((2 * I, H), "gu", wide / np.sqrt(H)), dn=bits((H, I), "dn", 1 / np.sqrt(I)),
                      dout=bits((T, H), "dout"), add=bits((T, H), "add") if add else None)
        self.bg = synth.normal_f32((2 * I,), 0.5, 0, "ffn_bg") if bias else None
        self.bd = synth.normal_f32((H,), 0.5, 0, "ffn_bd") if bias else None
        self.d = {k: None if v is None else _dev(v) for k, v in self.b.items()}
        dev = lambda v: None if v is None else torch.from_numpy(v).to(device())  # noqa: E731
        self.ffn = block.GluFfn(self.d["gu"], self.d["dn"], dev(self.bg), dev(self.bd), glu)
        f = {k: None if v is None else bf16.bf16_bits_to_f64(v) for k, v in self.b.items()}
        self.f = f
        bg, bd = (None if v is None else v.astype(np.float64) for v in (self.bg, self.bd))
        self.out, self.h, self.G = dense.ffn(f["x"], f["gu"], f["dn"], bg, bd, f["add"], glu)
        eacc = lambda K: (K / 16 + 2) * 2.0 ** -21  # noqa: E731
        g, u = self.G[:, :I], self.G[:, I:]
        dG0 = eacc(H) * (np.abs(f["x"]) @ np.abs(f["gu"]).T + (0 if bg is None else np.abs(bg)))
        ag, au = dense.act_grads(g, u, glu)
        e_h = (2 * (np.abs(ag) * dG0[:, :I] + np.abs(au) * dG0[:, I:]) + 1e-3 * dG0[:, :I] + 2.0 ** -18 * np.abs(self.h)
               + B8 * np.abs(self.h))
        e_out = e_h @ np.abs(f["dn"]).T + eacc(I) * (np.abs(self.h) @ np.abs(f["dn"]).T)
        self.e_out = e_out + B8 * (np.abs(self.out) + e_out) + 2.0 ** -20 * (0 if f["add"] is None else np.abs(f["add"]))
        self.grads = dense.ffn_backward(f["x"], f["gu"], f["dn"], f["dout"], bg, glu)
        dh = f["dout"] @ f["dn"]
        e_dh = eacc(H) * (np.abs(f["dout"]) @ np.abs(f["dn"]))
        curve = 1.2 * (np.abs(u) + (0 if glu is None else abs(glu[2])) + 1)
        slack = (dG0[:, :I] + dG0[:, I:]) * curve * np.abs(dh)
        e_g = np.concatenate([np.abs(ag) * e_dh + slack, np.abs(au) * e_dh + slack], axis=1)
        dG = np.concatenate([ag * dh, au * dh], axis=1)
        if glu:      # a value within its own error of a clamp may fall on either side of it
            edge = (np.abs(np.abs(self.G) - glu[1]) <= dG0)
            near = np.concatenate([edge[:, :I], edge[:, I:]], axis=1)
            e_g = e_g + near * np.concatenate([np.abs(dh) * curve, np.abs(dh) * (np.abs(g) + 1)], axis=1)
        e_g = e_g + 2.0 ** -18 * np.abs(dG)
        e_b = e_g + B8 * np.abs(dG)
        aG, ax, ad = np.abs(dG), np.abs(f["x"]), np.abs(f["dout"])
        e = [e_b @ np.abs(f["gu"]) + eacc(2 * I) * (aG @ np.abs(f["gu"])), e_b.T @ ax + eacc(T) * (aG.T @ ax),
             ad.T @ e_h + eacc(T) * (ad.T @ np.abs(self.h))]
        self.e_grads = [a + B8 * (np.abs(r) + a) for a, r in zip(e, self.grads[:3])]
        self.e_grads += [e_g.sum(0) + (T + 8) * 2.0 ** -24 * aG.sum(0), (T + 8) * 2.0 ** -24 * ad.sum(0)]

    def check_out(self, got):
        got = bf16_to_f64(got)
        assert np.isfinite(got).all() and (np.abs(got - self.out) <= self.e_out + 1e-30).all(), self._worst(got, self.out, self.e_out)
        assert np.linalg.norm(got - self.out) <= 5e-3 * np.linalg.norm(self.out) + 1e-30

    def check_grads(self, got):
        for name, v, r, e in zip(("dx", "dgu", "ddn", "dbg", "dbd"), got, self.grads, self.e_grads):
            if v is None:
                continue
            v = v.double().cpu().numpy()
            assert np.isfinite(v).all() and (np.abs(v - r) <= e + 1e-30).all(), (name, self._worst(v, r, e))
            assert np.linalg.norm(v - r) <= 1e-2 * np.linalg.norm(r) + 1e-30, name

    @staticmethod
    def _worst(v, r, e):
        i = np.unravel_index(np.argmax(np.abs(v - r) / (e + 1e-30)), v.shape)
        return f"at {i}: {v[i]} for {r[i]}, allowed {e[i]:.3g}; {np.mean(np.abs(v - r) > e):.3f} of all are off"


# tokens around the decode kernel's end, the tile height and its quarters; widths of one word, ragged against every
# tile width, and enough columns for the widest tile
SHAPES = [(1, 8, 8), (1, 2048, 768), (2, 64, 128), (7, 72, 200), (8, 264, 40), (9, 2048, 768), (16, 136, 1000),
          (17, 8, 8), (17, 64, 128), (31, 72, 200), (32, 200, 72), (33, 264, 776), (127, 512, 64), (128, 64, 512),
          (129, 128, 136), (300, 520, 296), (1000, 136, 2440), (700, 1400, 2808), (2050, 264, 1160),
          # each product of the pair in turn on CTA pairs, with ragged rows and columns
          (2050, 72, 2312), (2050, 2312, 72), (40, 2568, 2008),
          # narrower pair tiles, chosen where they fill the last wave
          (3300, 1800, 640), (3300, 640, 1800), (640, 3400, 1800)]


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_forward(T, H, I):
    for kw in (dict(), dict(glu=GLU, bias=True, add=True, wide=3.0)):
        c = Case(T, H, I, **kw)
        guard = torch.full((T + 3, H), 5.0, dtype=torch.bfloat16, device=device())
        out = c.ffn.forward(c.d["x"], c.d["add"], out=guard[:T])
        c.check_out(out)
        assert bool((guard[T:] == 5).all())
        if c.d["add"] is not None:                    # in place over the routed output
            acc = c.d["add"].clone()
            assert torch.equal(c.ffn.forward(c.d["x"], acc, out=acc), out)


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_training(T, H, I):
    for kw in (dict(add=True), dict(glu=GLU, bias=True, wide=3.0)):
        c = Case(T, H, I, **kw)
        out, saved = c.ffn.forward_train(c.d["x"], c.d["add"])
        c.check_out(out)
        grads = c.ffn.backward(saved, c.d["dout"])
        assert [g is None for g in grads] == [False] * 3 + [not kw.get("bias", False)] * 2
        c.check_grads(grads)
        assert e4b.e4b_device_status(saved.ws) == e4b.E4B_OK
        again = c.ffn.backward(saved, c.d["dout"])     # the same bits, and the saved state survives
        for a, b in zip(grads, again):
            assert (a is None and b is None) or torch.equal(a, b)
        only = c.ffn.backward(saved, c.d["dout"], weights=False)
        # (dx alone may run on another kernel than with the weight gradients: another order of the same sum)
        c.check_grads(only[:1])
        assert only[1:] == (None, None, None, None)


# one row of tiles of one CTA, 160, 192, 224 and 256 columns wide, for each of the three epilogues; two rows of them
@pytest.mark.parametrize("T,H,I", [(40, 72, 11400), (40, 72, 12288), (121, 72, 16000), (40, 72, 18904), (17, 72, 23000),
                                   (40, 72, 26008), (64, 72, 30000), (40, 72, 36000), (40, 23000, 72), (128, 26008, 72),
                                   (40, 30000, 72), (97, 36000, 72), (200, 72, 6000), (129, 11400, 72)])
def test_wide_tiles(T, H, I):
    c = Case(T, H, I, glu=GLU, bias=True, add=True)
    out, saved = c.ffn.forward_train(c.d["x"], c.d["add"])
    c.check_out(out)
    c.check_grads(c.ffn.backward(saved, c.d["dout"]))
    c.check_out(c.ffn.forward(c.d["x"], c.d["add"]))


# the products after dG in one launch on CTA pairs: ragged rows and columns, whole tiles, and two of the three
@pytest.mark.parametrize("T,H,I", [(509, 2048, 768), (512, 2560, 256), (513, 2600, 264), (1300, 1800, 648),
                                   (301, 2888, 2872), (2056, 1032, 1288)])
def test_grouped_gradients(T, H, I):
    c = Case(T, H, I, bias=True)
    out, saved = c.ffn.forward_train(c.d["x"])
    c.check_out(out)
    full = c.ffn.backward(saved, c.d["dout"])
    c.check_grads(full)
    for keep in ("110", "101", "011"):
        outs = [torch.full_like(t, 3.0) if k < 3 and keep[k] == "1" else None for k, t in enumerate(full)]
        e4b.e4b_ffn_backward(c.ffn.desc, T, c.d["x"], c.d["dout"], c.d["gu"], c.d["dn"], *outs, saved.ws)
        c.check_grads(outs)
    assert e4b.e4b_device_status(saved.ws) == e4b.E4B_OK


def test_each_gradient_alone():
    c = Case(40, 136, 72, bias=True)
    _, saved = c.ffn.forward_train(c.d["x"])
    full = c.ffn.backward(saved, c.d["dout"])
    for i in range(5):
        outs = [torch.full_like(t, 3.0) if k == i else None for k, t in enumerate(full)]
        e4b.e4b_ffn_backward(c.ffn.desc, 40, c.d["x"], c.d["dout"], c.d["gu"], c.d["dn"], *outs, saved.ws)
        c.check_grads(outs)


def test_no_tokens():
    c = Case(3, 64, 128, bias=True)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=device())
    assert c.ffn.forward(x).shape == (0, 64)
    out, saved = c.ffn.forward_train(x, x)
    assert e4b.e4b_device_status(saved.ws) == e4b.E4B_OK
    grads = c.ffn.backward(saved, x)
    assert grads[0].shape == (0, 64) and not any(bool(g.any()) for g in grads[1:])


def test_gradient_against_differences_of_the_definition():
    # sum(dout * out) along a random direction of every input, in fp64, against the kernel's gradients
    for glu in (None, GLU):
        c = Case(48, 64, 96, glu=glu, bias=True)
        _, saved = c.ffn.forward_train(c.d["x"])
        grads = [g.double().cpu().numpy() for g in c.ffn.backward(saved, c.d["dout"])]
        at = [c.f["x"], c.f["gu"], c.f["dn"], c.bg.astype(np.float64), c.bd.astype(np.float64)]
        for i in range(5):
            d = np.random.default_rng(i).standard_normal(at[i].shape)

            def loss(h):
                a = [v + h * d if k == i else v for k, v in enumerate(at)]
                return np.sum(c.f["dout"] * dense.ffn(a[0], a[1], a[2], a[3], a[4], glu=glu)[0])
            num = (loss(1e-6) - loss(-1e-6)) / 2e-6
            assert abs(np.sum(grads[i] * d) - num) <= np.sum(np.abs(d) * c.e_grads[i]) + 1e-6 * abs(num)


def test_two_forwards_before_their_backwards_and_other_streams():
    a, b = Case(40, 136, 72), Case(200, 136, 72)
    b.ffn = block.GluFfn(a.d["gu"], a.d["dn"])
    _, sa = a.ffn.forward_train(a.d["x"])
    _, sb = a.ffn.forward_train(b.d["x"])
    a.check_grads(a.ffn.backward(sa, a.d["dout"]))
    want = a.ffn.backward(sb, b.d["dout"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _, s = a.ffn.forward_train(b.d["x"])
        got = a.ffn.backward(s, b.d["dout"])
    torch.cuda.current_stream().wait_stream(side)
    for g, w in zip(got[:3], want[:3]):
        assert torch.equal(g, w)


@pytest.mark.parametrize("T", [4, 150])
def test_graphs_share_nothing_and_read_new_inputs(T):
    c = Case(T, 264, 136, glu=GLU, bias=True, add=True)
    c.ffn.forward(c.d["x"], c.d["add"])
    graphs, outs = [], []
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, saved = c.ffn.forward_train(c.d["x"], c.d["add"])
            grads = c.ffn.backward(saved, c.d["dout"])
        graphs.append(g)
        outs.append((out, grads, saved))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, grads, _ in outs:
        c.check_out(out)
        c.check_grads(grads)
    c.d["x"].zero_()
    graphs[0].replay()
    want = c.ffn.forward(c.d["x"], c.d["add"])
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want)


@pytest.mark.parametrize("T", [5, 40, 700])
@pytest.mark.parametrize("glu", [None, GLU])
def test_large_pre_activations_and_values_that_are_not_finite(T, glu):
    # gates of +-several hundred saturate the sigmoid; a NaN or an infinity of one token stays with that token
    c = Case(T, 136, 264, glu=glu, wide=60.0)
    assert np.abs(c.G).max() > 200
    out, saved = c.ffn.forward_train(c.d["x"])
    got = bf16_to_f64(out)
    assert np.isfinite(got).all() and np.linalg.norm(got - c.out) <= 5e-3 * np.linalg.norm(c.out)
    dx = bf16_to_f64(c.ffn.backward(saved, c.d["dout"])[0])
    assert np.isfinite(dx).all()
    x = c.d["x"].clone()
    x[2, 7], x[4, 100] = float("nan"), float("inf")
    out2, saved = c.ffn.forward_train(x)
    keep = [t for t in range(T) if t not in (2, 4)]
    assert torch.equal(out2[keep], out[keep])
    assert bool(torch.isnan(out2[2]).all())
    with np.errstate(all="ignore"):
        want = dense.ffn(x.double().cpu().numpy(), c.f["gu"], c.f["dn"], glu=glu)[0]
    assert np.array_equal(np.isnan(bf16_to_f64(out2)), np.isnan(want))
    dx2 = c.ffn.backward(saved, c.d["dout"])[0]
    assert torch.equal(dx2[keep], torch.from_numpy(dx).to(device()).bfloat16()[keep]) and bool(torch.isnan(dx2[2]).all())


def test_refusals():
    c = Case(20, 64, 128)
    x = c.d["x"]
    for bad in (x.float(), x[:, :32], x.t(), x[0], x.cpu()):
        with pytest.raises(ValueError):
            c.ffn.forward(bad)
    with pytest.raises(ValueError):
        c.ffn.forward(x, add=x[:2])
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        c.ffn.forward(x, out=x)
    with pytest.raises(ValueError):
        block.GluFfn(c.d["gu"][:-1], c.d["dn"])
    with pytest.raises(ValueError):
        block.GluFfn(c.d["gu"][:, :60].contiguous(), c.d["dn"][:60].contiguous())
    with pytest.raises(ValueError):
        block.GluFfn(c.d["gu"], c.d["dn"], glu=(1.0, -1.0, 0.0))
    _, saved = c.ffn.forward_train(x)
    with pytest.raises(ValueError):
        c.ffn.backward(saved, x[:3])
    odd = torch.zeros(20 * 64 + 1, dtype=torch.bfloat16, device=device())[1:].view(20, 64)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        c.ffn.forward(odd)

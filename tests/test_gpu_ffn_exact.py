"""The feed-forward block on data whose products add up without rounding: one non-zero value per row of x and of dout,
weights of few bits.  G and dh are then exact at every width, whatever kernel a token count takes, and a gate or up
exactly on a clamp passes its gradient (the ends count as inside).

Bias gradients: sum over t of dG, each term formed from exact G and dh.  The fast exponential is off by at most
2 + 1.173 |a g| ulp (16 for |a g| <= 12), the fast quotient by 2, so the sigmoid by 18 ulp, 2^-18.8 of its value; with
the few roundings that follow, 2^-17 of the sum of the magnitudes of the derivative's terms.  The sum over T terms in
fp32: (T + 8) 2^-24 of the magnitudes."""
import numpy as np
import pytest
import torch

from bit_mixture_experts_top_b200 import block
from helpers import bf16_to_f64, device
from oracle import dense

pytestmark = pytest.mark.gpu
GLU = (1.702, 7.0, 1.0)


def _case(T, H, I):
    g = np.random.default_rng(T + H)
    x, dout = np.zeros((T, H)), np.zeros((T, H))
    x[np.arange(T), 37 * np.arange(T) % H] = 1.0
    dout[np.arange(T), 53 * np.arange(T) % H] = 1.0
    gu = g.integers(-9, 10, (2 * I, H)).astype(np.float64)
    gu[g.random((2 * I, H)) < 0.3] = 7.0                      # many values exactly on a clamp, of either sign
    gu[g.random((2 * I, H)) < 0.1] = -7.0
    return x, gu, g.integers(-4, 5, (H, I)) / 4.0, dout


def _dev(a):
    return torch.from_numpy(a).to(device()).to(torch.bfloat16)


@pytest.mark.parametrize("glu", [GLU, None], ids=["clamped", "swiglu"])
@pytest.mark.parametrize("T,H,I", [(5, 2048, 72), (30, 2048, 72), (40, 2048, 72), (40, 12288, 72), (150, 2048, 264),
                                   (700, 2048, 264), (2050, 2048, 264), (2050, 4096, 1160), (40, 72, 12288)])
def test_exact_sums(T, H, I, glu):
    x, gu, dn, dout = _case(T, H, I)
    bg, bd = np.zeros(2 * I), np.zeros(H)
    f32 = lambda a: torch.from_numpy(a).float().to(device())  # noqa: E731
    ffn = block.GluFfn(_dev(gu), _dev(dn), f32(bg), f32(bd), glu)
    out, saved = ffn.forward_train(_dev(x))
    want, h, G = dense.ffn(x, gu, dn, glu=glu)
    # h is rounded once (2^-8), the sum over I may lose (I / 16 + 2) 2^-21, the output is rounded once
    slack = (np.abs(h) * (2.0 ** -8 + 2.0 ** -17 + (I / 16 + 2) * 2.0 ** -21)) @ np.abs(dn).T
    assert (np.abs(bf16_to_f64(out) - want) <= slack + 2.0 ** -8 * (np.abs(want) + slack)).all()
    got = ffn.backward(saved, _dev(dout))[3].double().cpu().numpy()
    g, u = G[:, :I], G[:, I:]
    ag, au = dense.act_grads(g, u, glu)
    dh = dout @ dn
    a, beta = (1.0, 0.0) if glu is None else (glu[0], glu[2])
    gc, uc = (g, u) if glu is None else (np.minimum(g, glu[1]), np.clip(u, -glu[1], glu[1]))
    s = 1 / (1 + np.exp(-a * gc))
    eg = np.abs((uc + beta) * s * (1 + a * np.abs(gc) * (1 - s)) * dh) * (ag != 0)
    eu = np.abs(gc * s * dh) * (au != 0)
    terms = np.concatenate([ag * dh, au * dh], axis=1)
    bound = 2.0 ** -17 * np.concatenate([eg, eu], axis=1).sum(0) + (T + 8) * 2.0 ** -24 * np.abs(terms).sum(0)
    off = np.abs(got - terms.sum(0))
    i = int(np.argmax(off - bound))
    assert (off <= bound + 1e-30).all(), (i, got[i], terms.sum(0)[i], bound[i], float(np.mean(off > bound)))

"""The kernels that only prompt and training sizes reach: the norm's forms for many rows (from 16 rows per SM on), the
norm backward's ring of row slots after it has wrapped several times, and column sums in several shares.

Tolerances are those of test_gpu_norm.py.  Forward: bit for bit, against the oracle where it is quick (all rows in bf16,
a sample of rows in 8 bits) and, for every row, against the same rows in calls of few rows, whose kernels
test_gpu_norm.py holds to the oracle.  Column sums: fp32 sums of T terms, (T + 8) 2^-24 of the magnitudes."""
import numpy as np
import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b
from helpers import device, to_np_bits
from oracle import bf16, dense
from test_gpu_norm import _bits, _check_backward, _dev, _inputs

pytestmark = pytest.mark.gpu
# the warp kernels (1, 2 and 4 words a lane) and the block kernels, at their borders and between
WIDTHS = [8, 96, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 2880, 2976, 3064, 3200, 4096]


def _rows(T):
    assert T >= 16 * torch.cuda.get_device_properties(0).multi_processor_count
    return T


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("residual", [True, False])
def test_forward_bits(H, residual):
    for T in (_rows(2401), 4100) if H == 2880 else (_rows(2401),):
        x, res, w = _inputs(T, H, residual)
        norm = block.RmsNorm(_dev(w), 1e-5)
        xd, rd = _dev(x), None if res is None else _dev(res)
        y, r, rstd = norm.forward_train(xd, rd)
        wr, ws, wy = dense.rmsnorm(x, res, w, 1e-5)
        assert np.array_equal(to_np_bits(r), wr) and np.array_equal(rstd.cpu().numpy(), ws)
        assert np.array_equal(to_np_bits(y), bf16.f64_to_bf16_bits(wy.astype(np.float64)))


@pytest.mark.parametrize("scales", ["mx", "row"])
@pytest.mark.parametrize("H", WIDTHS)
def test_8_bits(H, scales):
    if scales == "mx" and H % 32:
        pytest.skip("blocks of 32")
    T = _rows(2401)
    x, res, w = _inputs(T, H)
    x[5, H // 2], x[T - 2, H - 1] = 0x7F80, 0x7FC0        # an infinity, a NaN
    norm = block.RmsNorm(_dev(w), 1e-6)
    q, s, r = norm.forward_q8(_dev(x), _dev(res), scales=scales)
    q, s = q.view(torch.uint8), s.view(torch.uint8)
    for lo in range(0, T, 400):
        fq, fs, fr = norm.forward_q8(_dev(x[lo:lo + 400]), _dev(res[lo:lo + 400]), scales=scales)
        assert torch.equal(q[lo:lo + 400], fq.view(torch.uint8)) and torch.equal(r[lo:lo + 400].view(torch.int16), fr.view(torch.int16))
        few = fs.view(torch.uint8).reshape(-1)
        assert torch.equal(s.reshape(-1)[lo * len(few) // len(fq):][:len(few)], few)
    some = np.unique(np.r_[0:8, T - 8:T, np.random.default_rng(H).integers(0, T, 16)])
    _, _, wy = dense.rmsnorm(x[some], res[some], w, 1e-6)
    wq, wsc = (dense.quantize_mx if scales == "mx" else dense.quantize_rows)(wy)
    assert np.array_equal(q.cpu().numpy()[some], wq)
    got = s.reshape(T, -1)[torch.from_numpy(some).to(device())].cpu().numpy()
    assert np.array_equal(got if scales == "mx" else got.view(np.float32)[:, 0], wsc, equal_nan=scales == "row")


@pytest.mark.parametrize("H", [96, 2048, 2880, 4096])
def test_in_place(H):
    T = _rows(2401)
    x, res, w = _inputs(T, H)
    wr, _, wy = dense.rmsnorm(x, res, w, 1e-6)
    wb = bf16.f64_to_bf16_bits(wy.astype(np.float64))
    for swap in (False, True):
        xd, rd = _dev(x), _dev(res)
        r, y = (rd, xd) if swap else (xd, rd)
        e4b.e4b_rmsnorm(xd, rd, _dev(w), T, H, 1e-6, e4b.E4B_Q8_NONE, r, y, None, None, None)
        assert np.array_equal(to_np_bits(r), wr) and np.array_equal(to_np_bits(y), wb)


# (T, H): rows per group of threads far above the slots of its ring.  One and two words a thread with four slots, four
# with two, the widest rows with one (fp32 dy and dr together do not fit twice), each ragged against the groups
@pytest.mark.parametrize("T,H", [(20011, 8), (20011, 64), (20000, 256), (9001, 264), (9001, 512), (5003, 520), (5003, 1000),
                                 (5003, 2048), (5000, 2880), (3001, 4096), (1501, 8192), (601, 12288), (601, 16384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_ring(T, H, dtype):
    g = torch.Generator(device=device()).manual_seed(T + H)
    rand = lambda std, dt: (torch.randn(T, H, generator=g, device=device()) * std).to(dt)  # noqa: E731
    wb = _bits((H,), "mrw")
    w = bf16.bf16_bits_to_f64(wb)
    norm = block.RmsNorm(_dev(wb), 1e-3)
    r, dr, dy = rand(3.0, torch.bfloat16), rand(1.0, torch.bfloat16), rand(1.0, dtype)
    rstd = norm.forward_train(r)[2]
    for d in (dr, None):
        dx, dw = norm.backward(dy, r, rstd, d)
        _check_backward(dx, dw, dy, r, rstd, d, w)
        again = norm.backward(dy, r, rstd, d)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
        ws = torch.empty(e4b.e4b_rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=device())
        for target in (d, r) + ((dy,) if dtype == torch.bfloat16 else ()):
            if target is None:
                continue
            kept, dw2 = target.clone(), torch.empty_like(dw)
            e4b.e4b_rmsnorm_backward(dy, e4b.DTYPES[dtype], d, r, norm.weight, rstd, T, H, target, dw2, ws)
            assert torch.equal(target, dx) and torch.equal(dw2, dw)
            target.copy_(kept)
        assert e4b.e4b_device_status(ws) == e4b.E4B_OK


@pytest.mark.parametrize("T,H", [(1024, 72), (1025, 72), (3000, 136), (5000, 8), (140001, 8)])
def test_bias_gradients_in_several_shares(T, H):
    I = 8
    g = torch.Generator(device=device()).manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device=device()).to(torch.bfloat16)  # noqa: E731
    gu, dn, x, dout = rand(2 * I, H), rand(H, I), rand(T, H), rand(T, H)
    bias = [torch.zeros(n, device=device()) for n in (2 * I, H)]
    ffn = block.GluFfn(gu, dn, *bias)
    _, saved = ffn.forward_train(x)
    full = ffn.backward(saved, dout)
    want, mag = dout.double().sum(0), dout.double().abs().sum(0)
    alone = torch.full((H,), 3.0, device=device())
    e4b.e4b_ffn_backward(ffn.desc, T, x, dout, gu, dn, None, None, None, None, alone, saved.ws)
    for got in (alone, full[4]):
        assert bool(((got.double() - want).abs() <= (T + 8) * 2.0 ** -24 * mag).all())
    both = [torch.full((n,), 3.0, device=device()) for n in (2 * I, H)]
    e4b.e4b_ffn_backward(ffn.desc, T, x, dout, gu, dn, None, None, None, *both, saved.ws)
    assert torch.equal(both[1], alone)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    G = f(x) @ f(gu).T
    ag, au = dense.act_grads(G[:, :I], G[:, I:])
    dG = np.concatenate([ag, au], axis=1) * np.tile(f(dout) @ f(dn), (1, 2))
    # the sum itself, and 1e-4 for what test_gpu_ffn.py bounds: G, dh and the fast exponential (2^-18, K <= 136)
    assert (np.abs(f(both[0]) - dG.sum(0)) <= ((T + 8) * 2.0 ** -24 + 1e-4) * np.abs(dG).sum(0)).all()
    assert e4b.e4b_device_status(saved.ws) == e4b.E4B_OK

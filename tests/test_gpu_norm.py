"""GPU parity of the RMS norm (block.RmsNorm, e4b_rmsnorm, e4b_rmsnorm_backward) against oracle/dense.py.

Forward: bit for bit.  The stream is one bf16 rounding of an exact sum; the mean of squares is summed in fp64
on both sides, so rstd is the same fp32 value unless the fp64 sums fall on different sides of an fp32 rounding
border (their relative distance is below H 2^-53, the borders are 2^-24 apart); what follows is a fixed sequence
of single fp32 roundings.

Backward, |got - ref| per element, with u = 2^-24: dx = rstd (a - xh c) + dr is formed with at most 6 fp32
roundings on its terms, c is a sum of H products (at most H + 4 roundings, any order), and one rounding to bf16
of at most 2^-8.  dweight is a sum of T products of two rounded factors: at most (T + 3) u sum |dy xh|."""
import numpy as np
import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b, synth
from helpers import bf16_to_f64, device, to_np_bits
from oracle import bf16, dense

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _bits(shape, name, std=1.0):
    return synth.normal_bf16(shape, std, 0, name)


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device()).view(torch.bfloat16)


def _inputs(T, H, residual=True):
    x = _bits((T, H), f"nx{T}_{H}")
    res = _bits((T, H), f"nr{T}_{H}", 3.0) if residual else None
    w = _bits((H,), f"nw{H}")
    if T > 2:
        x[1] = 0
        if residual:
            res[1] = 0                      # a row of zeros
        x[2] = _bits((H,), "tiny", 2.0 ** -120)
    return x, res, w


# one value, one word, odd, ragged against the block width, each kernel's range and beyond it
SHAPES = [(1, 1), (3, 7), (5, 8), (4, 33), (3, 64), (17, 100), (1, 2048), (33, 2056), (7, 2880), (300, 96), (2, 8192),
          (3, 8200), (2, 32768), (2, 32776), (2, 40001), (9, 255), (5, 257), (400, 2883), (3, 8191), (3, 8193)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward_bits(T, H, residual):
    x, res, w = _inputs(T, H, residual)
    norm = block.RmsNorm(_dev(w), 1e-5)
    xd, rd = _dev(x), None if res is None else _dev(res)
    y, r, rstd = norm.forward_train(xd, rd)
    wr, ws, wy = dense.rmsnorm(x, res, w, 1e-5)
    assert np.array_equal(to_np_bits(r), wr)
    assert np.array_equal(rstd.cpu().numpy(), ws)
    assert np.array_equal(to_np_bits(y), bf16.f64_to_bf16_bits(wy.astype(np.float64)))
    y2, r2 = norm.forward(xd, rd)
    assert torch.equal(y2, y) and torch.equal(r2, r) and np.array_equal(to_np_bits(xd), x)
    if not residual:
        assert r.data_ptr() == xd.data_ptr()


@pytest.mark.parametrize("T,H", [(1, 32), (5, 96), (64, 2048), (9, 2880), (3, 8192), (2, 16384), (2, 32800)])
def test_mx_bits(T, H):
    x, res, w = _inputs(T, H)
    q, s, r = block.RmsNorm(_dev(w), 1e-6).forward_q8(_dev(x), _dev(res), scales="mx")
    wr, _, wy = dense.rmsnorm(x, res, w, 1e-6)
    wq, ws = dense.quantize_mx(wy)
    assert q.dtype == torch.float8_e4m3fn and np.array_equal(to_np_bits(r), wr)
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.view(torch.uint8).cpu().numpy(), wq)


@pytest.mark.parametrize("T,H", [(1, 1), (5, 33), (64, 2048), (9, 2880), (3, 8192), (2, 32768), (2, 40001)])
def test_row_scale_bits(T, H):
    x, _, w = _inputs(T, H, False)
    q, s, _ = block.RmsNorm(_dev(w), 1e-6).forward_q8(_dev(x), scales="row")
    wq, ws = dense.quantize_rows(dense.rmsnorm(x, None, w, 1e-6)[2])
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.view(torch.uint8).cpu().numpy(), wq)


@pytest.mark.parametrize("H", [96, 33 * 32, 32800])
def test_values_that_are_not_finite_stay_in_their_row(H):
    x, _, w = _inputs(6, H, False)
    x[2, 5], x[4, 40] = 0x7F80, 0x7FC0                     # an infinity, a NaN
    norm = block.RmsNorm(_dev(w), 1e-6)
    _, _, wy = dense.rmsnorm(x, None, w, 1e-6)
    y, _ = norm.forward(_dev(x))
    got = bf16_to_f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(wy)) and np.isfinite(got[[0, 1, 3, 5]]).all()
    for scales, want in (("row", dense.quantize_rows(wy)), ("mx", dense.quantize_mx(wy))):
        q, s, _ = norm.forward_q8(_dev(x), scales=scales)
        assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want[0]), scales
        assert np.array_equal(s.cpu().numpy(), want[1], equal_nan=scales == "row"), scales


def test_in_place_and_both_outputs_at_once():
    for T, H in ((5, 2880), (5, 33 * 32 + 32), (3, 40000)):
        x, res, w = _inputs(T, H)
        wr, _, wy = dense.rmsnorm(x, res, w, 1e-6)
        wq, ws = dense.quantize_mx(wy)
        for target in ("x", "res"):
            xd, rd, wd = _dev(x), _dev(res), _dev(w)
            # the stream replaces the residual (or x), the normed rows the other one
            r, y = (xd, rd) if target == "x" else (rd, xd)
            q = torch.empty((T, H), dtype=torch.uint8, device=device())
            s = torch.empty((T, H // 32), dtype=torch.uint8, device=device())
            e4b.e4b_rmsnorm(xd, rd, wd, T, H, 1e-6, e4b.E4B_Q8_MX, r, y, q, s, None)
            assert np.array_equal(to_np_bits(r), wr), (target, H)
            assert np.array_equal(to_np_bits(y), bf16.f64_to_bf16_bits(wy.astype(np.float64))), (target, H)
            assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


@pytest.mark.parametrize("shift", [1, 3, 4])
def test_misaligned_rows(shift):
    T, H = 4, 256
    x, res, w = _inputs(T, H)
    buf = torch.zeros(T * H + 8, dtype=torch.bfloat16, device=device())
    xd = buf[shift:shift + T * H].view(T, H)
    xd.copy_(_dev(x))
    y, r = block.RmsNorm(_dev(w)).forward(xd, _dev(res))
    wr, _, wy = dense.rmsnorm(x, res, w, 1e-6)
    assert np.array_equal(to_np_bits(r), wr)
    assert np.array_equal(to_np_bits(y), bf16.f64_to_bf16_bits(wy.astype(np.float64)))


@pytest.mark.parametrize("H", [32, 256, 2880, 8192, 8224])
def test_misaligned_rows_in_8_bits(H):
    T = 4
    x, res, w = _inputs(T, H)
    x[1, 7], x[2, 31] = 0x7F80, 0x7FC0                     # an infinity, a NaN
    buf = torch.zeros(T * H + 8, dtype=torch.bfloat16, device=device())
    xd = buf[3:3 + T * H].view(T, H)
    xd.copy_(_dev(x))
    _, _, wy = dense.rmsnorm(x, res, w, 1e-6)
    for scales, want in (("row", dense.quantize_rows(wy)), ("mx", dense.quantize_mx(wy))):
        q, s, _ = block.RmsNorm(_dev(w)).forward_q8(xd, _dev(res), scales=scales)
        assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want[0]), scales
        assert np.array_equal(s.cpu().numpy(), want[1], equal_nan=scales == "row"), scales


@pytest.mark.parametrize("H", [64, 2048, 2056, 4096, 8200, 33])
def test_subnormals_and_signed_zeros(H):
    g = np.random.default_rng(H)
    sub = lambda: (g.integers(0, 0x80, (4, H)) | (g.integers(0, 2, (4, H)) << 15)).astype(np.uint16)  # noqa: E731
    x, res, w = sub(), sub(), _bits((H,), "sw")
    res[1] = x[1] ^ 0x8000                                # sums that cancel
    res[2], x[2] = 0x8000, 0x8000                         # -0 + -0
    for eps in (0.0, 1e-30, 1e-6):
        norm = block.RmsNorm(_dev(w), eps)
        y, r, rstd = norm.forward_train(_dev(x), _dev(res))
        wr, ws, wy = dense.rmsnorm(x, res, w, eps)
        assert np.array_equal(to_np_bits(r), wr) and np.array_equal(rstd.cpu().numpy(), ws)
        fine = np.isfinite(wy)                            # a row of zeros without eps is 0 * inf
        assert np.array_equal(to_np_bits(y)[fine], bf16.f64_to_bf16_bits(wy.astype(np.float64))[fine])
        assert np.isnan(bf16_to_f64(y)[~fine]).all()
        q, s, _ = norm.forward_q8(_dev(x), _dev(res), scales="row")
        wq, wsc = dense.quantize_rows(wy)
        assert np.array_equal(q.view(torch.uint8).cpu().numpy(), wq)
        assert np.array_equal(s.cpu().numpy(), wsc, equal_nan=True)


@pytest.mark.parametrize("H", [64, 2056, 33])
def test_values_whose_squares_leave_the_fp32_range(H):
    x, _, w = _inputs(5, H, False)
    x[0] = _bits((H,), "huge", 2.0 ** 100)
    x[3] = _bits((H,), "small", 2.0 ** -100)
    norm = block.RmsNorm(_dev(w), 0.0)
    y, r, rstd = norm.forward_train(_dev(x))
    _, ws, wy = dense.rmsnorm(x, None, w, 0.0)
    fine = np.isfinite(wy)
    assert fine[[0, 2, 3, 4]].all() and np.array_equal(rstd.cpu().numpy(), ws)
    assert np.array_equal(to_np_bits(y)[fine], bf16.f64_to_bf16_bits(wy.astype(np.float64))[fine])


def test_no_rows():
    norm = block.RmsNorm(_dev(_bits((64,), "w")))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=device())
    y, r, rstd = norm.forward_train(x, x.clone())
    assert y.shape == (0, 64) and r.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = norm.backward(x.float(), r, rstd)
    assert dx.shape == (0, 64) and not dw.any() and dw.shape == (64,)


def _backward_case(T, H, dtype, with_dr, shift=0):
    x, res, w = _inputs(T, H)
    norm = block.RmsNorm(_dev(w), 1e-3)
    _, r, rstd = norm.forward_train(_dev(x), _dev(res))
    g = np.random.default_rng(T * H)
    dy = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(device()).to(dtype)
    dr = _dev(_bits((T, H), "dr")) if with_dr else None
    if shift:
        flat = torch.zeros(T * H + shift, dtype=dtype, device=device())
        flat[shift:] = dy.flatten()
        dy = flat[shift:].view(T, H)
    return norm, dy, r, rstd, dr, bf16.bf16_bits_to_f64(w)


def _check_backward(dx, dw, dy, r, rstd, dr, w):
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    dy, r, rstd, dr = f(dy), f(r), f(rstd), f(dr)
    T, H = r.shape
    wdx, wdw = dense.rmsnorm_backward(dy, r, w, rstd, dr)
    a, xh = np.abs(dy * w), np.abs(r * rstd[:, None])
    mean = np.mean(a * xh, axis=1, keepdims=True)
    terms = rstd[:, None] * (a + xh * mean) + (0 if dr is None else np.abs(dr))
    err = 6 * U * terms + (H + 4) * U * rstd[:, None] * xh * mean
    assert (np.abs(f(dx) - wdx) <= 2.0 ** -8 * (np.abs(wdx) + err) + err + 1e-38).all()
    assert (np.abs(f(dw) - wdw) <= (T + 3) * U * np.sum(np.abs(dy) * xh, axis=0) + 1e-38).all()


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 64), (5, 2048), (37, 2880), (1000, 96), (4, 4096), (9, 4104), (6, 8192),
                                 (5, 16384), (3, 16392), (11, 1001), (700, 4096)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(T, H, dtype):
    for with_dr in (True, False):
        norm, dy, r, rstd, dr, w = _backward_case(T, H, dtype, with_dr)
        dx, dw = norm.backward(dy, r, rstd, dr)
        _check_backward(dx, dw, dy, r, rstd, dr, w)
        again = norm.backward(dy, r, rstd, dr)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_backward_misaligned_and_in_place():
    norm, dy, r, rstd, dr, w = _backward_case(6, 512, torch.float32, True, shift=1)
    dx, dw = norm.backward(dy, r, rstd, dr)
    _check_backward(dx, dw, dy, r, rstd, dr, w)
    for H in (512, 33):                       # the gradient of the stream replaced by dx, on both kernels
        for dt in (torch.float32, torch.bfloat16):
            norm, dy, r, rstd, dr, w = _backward_case(6, H, dt, True)
            dx, dw = norm.backward(dy, r, rstd, dr)
            targets = [dr, r] + ([dy] if dt == torch.bfloat16 else [])
            for target in targets:
                kept = target.clone()
                dw2 = torch.empty_like(dw)
                ws = torch.empty(e4b.e4b_rmsnorm_backward_workspace_bytes(6, H), dtype=torch.uint8, device=device())
                e4b.e4b_rmsnorm_backward(dy, e4b.DTYPES[dt], dr, r, norm.weight, rstd, 6, H, target, dw2, ws)
                assert torch.equal(target, dx) and torch.equal(dw2, dw)
                target.copy_(kept)


def test_gradient_against_differences():
    # the kernel's own forward in fp32 rows: sum(dy * y) along a direction, against <dx, direction>
    T, H = 3, 512
    x = _dev(_bits((T, H), "fd_x"))
    w = _dev(_bits((H,), "fd_w"))
    norm = block.RmsNorm(w, 1e-3)
    dy = torch.from_numpy(np.random.default_rng(0).standard_normal((T, H)).astype(np.float32)).to(device())
    _, r, rstd = norm.forward_train(x)
    dx, dw = norm.backward(dy, r, rstd)

    def loss(xv):          # the definition in fp64 at any x
        rs = 1 / torch.sqrt(xv.square().mean(1, keepdim=True) + 1e-3)
        return (dy.double() * xv * rs * w.double()).sum()
    d = torch.randn(T, H, generator=torch.Generator().manual_seed(1), dtype=torch.float64).to(device())
    h = 1e-5
    num = (loss(x.double() + h * d) - loss(x.double() - h * d)) / (2 * h)
    # dx carries bf16 roundings of at most 2^-8 each (rstd's fp32 rounding and h^2 are far below)
    assert abs(float((dx.double() * d).sum() - num)) <= 2.0 ** -8 * float((dx.double() * d).abs().sum())


def test_streams_and_graph_replay_read_new_inputs():
    T, H = 33, 2880
    x, res, w = _inputs(T, H)
    norm = block.RmsNorm(_dev(w))
    xd, rd = _dev(x), _dev(res)
    want_y, want_r = norm.forward(xd, rd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, r = norm.forward(xd, rd)
        dx, dw = norm.backward(y, r, norm.forward_train(xd, rd)[2])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want_y) and torch.equal(r, want_r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gy, gr, gs = norm.forward_train(xd, rd)
        gdx, gdw = norm.backward(gy, gr, gs)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gy, want_y) and torch.equal(gdx, dx) and torch.equal(gdw, dw)
    xd.mul_(-2)
    want_y, want_r = norm.forward(xd, rd)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gy, want_y) and torch.equal(gr, want_r)


def test_refusals():
    norm = block.RmsNorm(_dev(_bits((64,), "w")))
    x = _dev(_bits((4, 64), "x"))
    for bad in (x[:, :32], x.float(), x.t(), x[0], x.cpu()):
        with pytest.raises(ValueError):
            norm.forward(bad)
    with pytest.raises(ValueError):
        norm.forward(x, x[:2])
    with pytest.raises(ValueError, match="contiguous"):
        norm.forward(torch.empty((64, 4), dtype=torch.bfloat16, device=device()).t())
    with pytest.raises(ValueError, match="scales"):
        norm.forward_q8(x, scales="tensor")
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        block.RmsNorm(_dev(_bits((40,), "w40"))).forward_q8(_dev(_bits((4, 40), "x40")))
    _, r, rstd = norm.forward_train(x)
    with pytest.raises(ValueError):
        norm.backward(x.half(), r, rstd)
    with pytest.raises(ValueError):
        norm.backward(x, r, rstd[:3])

"""CPU oracle of the dense operators around the routed layer (test infrastructure only): the RMS norm with
the residual's addition, its 8-bit outputs and its backward; the gated feed-forward block and its backward;
the global gradient norm with clipping.

fp64 throughout, except where the operator's definition fixes a precision: the stream r is bf16, rstd and
the normed value before its last rounding are fp32 (so that the 8-bit codes are defined bit for bit).
"""
import numpy as np

from . import bf16


def e4m3_values():
    """The 127 non-negative finite e4m3 values in code order (code 0x7F is NaN): 4 exponent bits, bias 7, 3
    mantissa bits, subnormals, largest 448."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


def round_to_e4m3(x):
    """e4m3 codes (uint8) of float64 values with |x| <= 448, nearest, ties to the even code; NaN gives 0x7F."""
    v = e4m3_values()
    mid = (v[1:] + v[:-1]) / 2
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    lo = np.searchsorted(mid, a, side="left")            # midpoints strictly below a
    hi = np.searchsorted(mid, a, side="right")
    code = np.where((lo != hi) & (lo % 2 == 1), hi, lo)   # a tie sits between codes lo and lo + 1
    code = np.where(np.isnan(x), 0x7F, code | (np.signbit(x).astype(np.int64) << 7))
    return code.astype(np.uint8)


def rmsnorm(x_bits, residual_bits, weight_bits, eps):
    """(r bf16 bits, rstd fp32, y fp32): y is the value that the bf16 and 8-bit outputs round."""
    r_bits = np.asarray(x_bits, np.uint16)
    if residual_bits is not None:
        r_bits = bf16.f64_to_bf16_bits(bf16.bf16_bits_to_f64(x_bits) + bf16.bf16_bits_to_f64(residual_bits))
    r = bf16.bf16_bits_to_f64(r_bits)
    with np.errstate(all="ignore"):
        rstd = (1.0 / np.sqrt(np.mean(r * r, axis=1) + eps)).astype(np.float32)
        y = r.astype(np.float32) * rstd[:, None]
        y = y * bf16.bf16_bits_to_f64(weight_bits).astype(np.float32)
    return r_bits, rstd, y


def quantize_rows(y):
    """(e4m3 codes, fp32 scale per row) of fp32 rows."""
    y = np.asarray(y, np.float32)
    q = np.empty(y.shape, np.uint8)
    s = np.empty(y.shape[0], np.float32)
    for t, row in enumerate(y):
        if not np.all(np.isfinite(row)):
            q[t], s[t] = 0x7F, np.nan
            continue
        s[t] = max(np.float32(np.abs(row).max() / np.float32(448)), np.float32(2.0 ** -126))
        q[t] = round_to_e4m3((row / s[t]).astype(np.float64))
    return q, s


def quantize_mx(y):
    """(e4m3 codes, E8M0 bytes per 32 values) of fp32 rows whose length is a multiple of 32."""
    y = np.asarray(y, np.float32)
    T, H = y.shape
    blocks = y.reshape(-1, 32).astype(np.float64)
    q = np.empty(blocks.shape, np.uint8)
    s = np.empty(len(blocks), np.uint8)
    for i, b in enumerate(blocks):
        if not np.all(np.isfinite(b)):
            q[i], s[i] = 0x7F, 255
            continue
        e = -127
        while np.abs(b).max() > 448.0 * 2.0 ** e:
            e += 1
        s[i] = e + 127
        q[i] = round_to_e4m3(b * 2.0 ** -e)
    return q.reshape(T, H), s.reshape(T, H // 32)


def rmsnorm_backward(dy, r, weight, rstd, dr=None):
    """(dx, dweight) of sum(dy * y) + sum(dr * r), all float64."""
    xh = r * rstd[:, None]
    a = dy * weight
    dx = rstd[:, None] * (a - xh * np.mean(a * xh, axis=1, keepdims=True))
    if dr is not None:
        dx = dx + dr
    return dx, np.sum(dy * xh, axis=0)


def act(g, u, glu=None):
    """silu(g) * u, or the clamped GLU with glu = (alpha, limit, beta)."""
    if glu is None:
        return g / (1.0 + np.exp(-g)) * u
    alpha, limit, beta = glu
    g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    return g / (1.0 + np.exp(-alpha * g)) * (u + beta)


def act_grads(g, u, glu=None):
    """d act / d g and d act / d u; the clamps pass the gradient inside their range, ends included."""
    if glu is None:
        s = 1.0 / (1.0 + np.exp(-g))
        return u * (s + g * s * (1.0 - s)), g * s
    alpha, limit, beta = glu
    gc, uc = np.minimum(g, limit), np.clip(u, -limit, limit)
    s = 1.0 / (1.0 + np.exp(-alpha * gc))
    dg = (s + alpha * gc * s * (1.0 - s)) * (uc + beta)
    return np.where(g > limit, 0.0, dg), np.where((u < -limit) | (u > limit), 0.0, gc * s)


def ffn(x, w_gu, w_dn, gu_bias=None, dn_bias=None, add=None, glu=None):
    """(out, h, G): out = act(x W_gate^T, x W_up^T) W_dn^T + add, with biases; w_gu [2I, H], w_dn [H, I]."""
    I = w_dn.shape[1]
    G = x @ w_gu.T + (0.0 if gu_bias is None else gu_bias)
    h = act(G[:, :I], G[:, I:], glu)
    out = h @ w_dn.T + (0.0 if dn_bias is None else dn_bias) + (0.0 if add is None else add)
    return out, h, G


def ffn_backward(x, w_gu, w_dn, dout, gu_bias=None, glu=None):
    """Gradients of sum(dout * out): (dx, dw_gu, dw_dn, dgu_bias, ddn_bias)."""
    I = w_dn.shape[1]
    _, h, G = ffn(x, w_gu, w_dn, gu_bias, glu=glu)
    dh = dout @ w_dn
    dg, du = act_grads(G[:, :I], G[:, I:], glu)
    dG = np.concatenate([dg * dh, du * dh], axis=1)
    return dG @ w_gu, dG.T @ x, dout.T @ h, dG.sum(axis=0), dout.sum(axis=0)


def clip_grads(grads, max_norm):
    """(norm, clipped float64 arrays) of a list of float64 arrays."""
    norm = float(np.sqrt(sum(float(np.sum(g * g)) for g in grads)))
    c = 1.0 if np.isinf(max_norm) else min(1.0, max_norm / (norm + 1e-6))
    return norm, [g * c for g in grads]

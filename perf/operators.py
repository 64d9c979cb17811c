"""The dense operators around the routed 4-bit layer, as cases to measure: the RMS norm with the residual's
addition (bf16 or 8-bit output, and its backward), the gated feed-forward block of a shared expert (forward,
and a training step's forward and backward), and the global gradient norm with clipping.

``run`` computes a case in plain torch operations, or with ``own`` through the package's classes."""
import math

import numpy as np
import torch

own = False

GLU = (1.702, 7.0, 1.0)     # clamped GLU constants of the layer's gpt-oss epilogue


def listed():
    return [
        # one token's norm before the layer, Qwen3-30B-A3B-shaped: launch latency
        dict(name="norm_decode_1", op="norm", T=1, H=2048, residual=True, eps=1e-6),
        # a decode batch whose normed rows go out in 8 bits with one scale per row
        dict(name="norm_row8_decode_64", op="norm_q8", T=64, H=2048, residual=True, scales="row", eps=1e-6),
        # prefill of a gpt-oss-shaped layer, ragged token count, 8 bits with a power-of-two scale per 32 values
        dict(name="norm_mx8_prefill_4099", op="norm_q8", T=4099, H=2880, residual=True, scales="mx", eps=1e-5),
        # the norm's backward in a training step; dy is the routed layer's fp32 input gradient
        dict(name="norm_backward_16384", op="norm_backward", T=16384, H=2880, dy="f32", dr=True),
        # the shared expert for a single token: weight stream and launch latency
        dict(name="ffn_decode_1", op="ffn", T=1, H=2048, I=768, glu=False, bias=False, add=True),
        # a decode batch, gpt-oss-shaped with biases and the clamped GLU
        dict(name="ffn_decode_64", op="ffn", T=64, H=2880, I=2880, glu=True, bias=True, add=True),
        # prefill, gpt-oss-shaped
        dict(name="ffn_prefill_4096", op="ffn", T=4096, H=2880, I=2880, glu=True, bias=True, add=True),
        # a training step of the shared expert at the fine-tuning batch of the LoRA workload, ragged, with biases
        dict(name="ffn_train_509", op="ffn_train", T=509, H=2048, I=768, glu=False, bias=True, add=True),
        # a training step of a large dense block: tensor-core bound
        dict(name="ffn_train_8192", op="ffn_train", T=8192, H=4096, I=12288, glu=False, bias=False, add=False),
        # the adapter gradients of one Qwen3-30B-A3B-shaped layer
        dict(name="clip_layer", op="clip", tensors=2, mean=1835008, shape_seed=0, mix="f32", packed=False, max_norm=1.0),
        # the adapter gradients of a whole model of such layers
        dict(name="clip_model", op="clip", tensors=96, mean=1835008, shape_seed=0, mix="f32", packed=False, max_norm=1.0),
        # many tensors of all sizes and types, packed one after the other without alignment
        dict(name="clip_mixed_401", op="clip", tensors=401, mean=90000, shape_seed=7, mix="all", packed=True,
             max_norm=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_q8", "norm_backward", "ffn", "ffn", "ffn_train", "clip"])
    if op.startswith("norm"):
        T, H = _log(rng, 1, 16384), _log(rng, 32, 8192)
        if rng.random() < 0.7:
            H = max(32, H // 32 * 32)
        T = max(1, min(T, 16384 * 2880 // H))
        if op == "norm_backward":
            return dict(op=op, T=T, H=H, dy=rng.choice(["f32", "bf16"]), dr=rng.random() < 0.7)
        c = dict(op=op, T=T, H=H, residual=rng.random() < 0.7, eps=rng.choice([1e-5, 1e-6]))
        if op == "norm_q8":
            c["scales"] = "row" if H % 32 else rng.choice(["row", "mx"])
        return c
    if op.startswith("ffn"):
        H, I = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 1536)
        T = min(_log(rng, 1, 8192), 8192 * 4096 * 12288 // (H * I))
        # fp32 bias gradients inherit the tensor cores' accumulation error, 1.1e-9 per product in the sum over H
        bias = rng.random() < 0.5 and (op == "ffn" or H <= 2048)
        return dict(op=op, T=T, H=H, I=I, glu=rng.random() < 0.5, bias=bias, add=rng.random() < 0.5)
    n = _log(rng, 1, 600)
    return dict(op=op, tensors=n, mean=_log(rng, 10, min(2000000, 170000000 // n)), shape_seed=rng.randrange(1 << 20),
                mix=rng.choice(["f32", "bf16", "all"]), packed=rng.random() < 0.5,
                max_norm=rng.choice([0.1, 1.0, 1e6]))


# ---------------------------------------------------------------------------- inputs

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _clip_shapes(case):
    """[(type, elements)] of a clip case.  Seed 0 is the layer's own pair of adapter gradients (dA of
    128 x 2048 x 8 and dB of 128 x 8 x 1536), repeated; other seeds draw sizes and types."""
    n = case["tensors"]
    if case["shape_seed"] == 0:
        return [("f32", 128 * 2048 * 8 if i % 2 == 0 else 128 * 8 * 1536) for i in range(n)]
    g = np.random.Generator(np.random.PCG64(case["shape_seed"]))
    sizes = np.exp(g.normal(0.0, 1.5, size=n))
    sizes = np.maximum(1, sizes * (case["mean"] * n / sizes.sum())).astype(np.int64)
    names = ["f32", "bf16", "f16"] if case["mix"] == "all" else [case["mix"]]
    return [(names[int(i)], int(s)) for i, s in zip(g.integers(0, len(names), size=n), sizes)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s = {"case": case}
    if case["op"] in ("norm", "norm_q8", "norm_backward"):
        T, H = case["T"], case["H"]
        channel = torch.exp(0.5 * torch.randn(H, generator=g, device=dev))     # some channels far larger than others
        s["weight"] = (1.0 + 0.2 * torch.randn(H, generator=g, device=dev)).to(torch.bfloat16)
        if case["op"] == "norm_backward":
            s["r"] = (normal(T, H, dtype=torch.float32) * channel).to(torch.bfloat16)
            s["rstd"] = (1.0 / (s["r"].double().square().mean(dim=1) + 1e-6).sqrt()).float()
            s["dy"] = normal(T, H, std=0.01, dtype=_TYPES[case["dy"]])
            s["dr"] = normal(T, H, std=0.01) if case["dr"] else None
        else:
            s["x"] = normal(T, H, std=0.5)
            s["residual"] = (normal(T, H, dtype=torch.float32) * channel).to(torch.bfloat16) if case["residual"] else None
        if own:
            from bit_mixture_experts_top_b200 import block
            s["norm"] = block.RmsNorm(s["weight"], case.get("eps", 1e-6))
    elif case["op"] in ("ffn", "ffn_train"):
        T, H, I = case["T"], case["H"], case["I"]
        s["x"] = normal(T, H)
        s["gate_up"] = normal(2 * I, H, std=1.0 / math.sqrt(H))
        s["down"] = normal(H, I, std=1.0 / math.sqrt(I))
        s["gu_bias"] = normal(2 * I, std=0.2, dtype=torch.float32) if case["bias"] else None
        s["dn_bias"] = normal(H, std=0.2, dtype=torch.float32) if case["bias"] else None
        s["add"] = normal(T, H) if case["add"] else None
        s["dout"] = normal(T, H, std=0.01) if case["op"] == "ffn_train" else None
        if own:
            from bit_mixture_experts_top_b200 import block
            s["ffn"] = block.GluFfn(s["gate_up"], s["down"], s["gu_bias"], s["dn_bias"], GLU if case["glu"] else None)
    else:
        shapes = _clip_shapes(case)
        s["flat"], s["clipped"], grads, outs = {}, {}, [], []
        align = 1 if case["packed"] else 128
        start, at = {k: 0 for k in _TYPES}, []
        for name, n in shapes:
            at.append(start[name])
            start[name] += (n + align - 1) // align * align
        for name, n in start.items():
            if n:
                s["flat"][name] = normal(n, dtype=torch.float32).mul_(0.02).to(_TYPES[name])
                s["clipped"][name] = torch.zeros(n, dtype=_TYPES[name], device=dev)
        for (name, n), a in zip(shapes, at):
            end = (a + n + align - 1) // align * align
            s["flat"][name][a + n:end] = 0
            grads.append(s["flat"][name][a:a + n])
            outs.append(s["clipped"][name][a:a + n])
        if own:
            from bit_mixture_experts_top_b200 import block
            s["clipper"] = block.GradClipper(grads, outs)
    return s


# ---------------------------------------------------------------------------- one pass

def _plain_norm(s):
    x, w = s["x"], s["weight"].float()
    r = x if s["residual"] is None else (x.float() + s["residual"].float()).to(torch.bfloat16)
    # the mean of squares in 64 bits, so that an 8-bit value next to a rounding border has one answer
    rstd = (1.0 / torch.sqrt(r.double().square().mean(dim=1, keepdim=True) + s["case"]["eps"])).float()
    return r, r.float() * rstd * w


def _plain_q8(y, scales):
    amax = y.abs()
    if scales == "row":
        scale = torch.clamp(amax.amax(dim=1) / 448.0, min=2.0 ** -126)
        return (y / scale[:, None]).to(torch.float8_e4m3fn), scale
    T, H = y.shape
    m, e = torch.frexp(amax.reshape(T, H // 32, 32).amax(dim=2))      # amax = m 2^e, 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    byte = torch.where(m == 0, torch.zeros_like(e), torch.clamp(e + 127, 0, 254))
    q = torch.ldexp(y.reshape(T, H // 32, 32).double(), (127 - byte)[:, :, None].double()).float()
    return q.reshape(T, H).to(torch.float8_e4m3fn), byte.to(torch.uint8)


def _plain_act(g, u, glu):
    if glu:
        alpha, limit, beta = GLU
        g, u = torch.clamp(g, max=limit), torch.clamp(u, -limit, limit)
        return g * torch.sigmoid(alpha * g) * (u + beta)
    return g * torch.sigmoid(g) * u


def _plain_act_grads(g, u, glu):
    if glu:
        alpha, limit, beta = GLU
        gc, uc = torch.clamp(g, max=limit), torch.clamp(u, -limit, limit)
        sg = torch.sigmoid(alpha * gc)
        dg = sg * (1 + alpha * gc * (1 - sg)) * (uc + beta) * (g <= limit)
        return dg, gc * sg * ((u >= -limit) & (u <= limit))
    sg = torch.sigmoid(g)
    return u * sg * (1 + g * (1 - sg)), g * sg


def _plain_ffn(s, train):
    case, bf16 = s["case"], torch.bfloat16
    I = case["I"]
    x, wgu, wdn = s["x"].float(), s["gate_up"].float(), s["down"].float()
    G = x @ wgu.t()
    if case["bias"]:
        G = G + s["gu_bias"]
    g, u = G[:, :I], G[:, I:]
    h = _plain_act(g, u, case["glu"])
    out = h @ wdn.t()
    if case["bias"]:
        out = out + s["dn_bias"]
    if case["add"]:
        out = out + s["add"].float()
    out = out.to(bf16)
    if not train:
        return out
    dout = s["dout"].float()
    dh = dout @ wdn
    dg, du = _plain_act_grads(g, u, case["glu"])
    dG = torch.cat([dg * dh, du * dh], dim=1)
    got = [out, (dG @ wgu).to(bf16), (dG.t() @ x).to(bf16), (dout.t() @ h).to(bf16)]
    if case["bias"]:
        got += [dG.sum(dim=0, dtype=torch.float64).float(), dout.sum(dim=0, dtype=torch.float64).float()]
    return got


def _plain_norm_backward(s):
    r, w, rstd, dy = s["r"].float(), s["weight"].float(), s["rstd"][:, None], s["dy"].float()
    xh = r * rstd
    c = (dy * w * xh).sum(dim=1, keepdim=True, dtype=torch.float64) / s["case"]["H"]
    dx = rstd * (dy * w - xh * c.float())
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return dx.to(torch.bfloat16), (dy * xh).sum(dim=0, dtype=torch.float64).float()


def _plain_clip(s):
    sums = [f.float().square().sum(dtype=torch.float64) for f in s["flat"].values()]
    norm = torch.stack(sums).sum().sqrt()
    c = torch.clamp(s["case"]["max_norm"] / (norm + 1e-6), max=1.0).float()
    return [norm.float()] + [(f.float() * c).to(f.dtype) for f in s["flat"].values()]


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        if own:
            y, r = s["norm"].forward(s["x"], s["residual"])
        else:
            r, y = _plain_norm(s)
            y = y.to(torch.bfloat16)
        return {"y": y, "r": r}
    if op == "norm_q8":
        if own:
            q, scales, r = s["norm"].forward_q8(s["x"], s["residual"], scales=case["scales"])
        else:
            r, y = _plain_norm(s)
            q, scales = _plain_q8(y, case["scales"])
        return {"q": q, "scales": scales, "r": r}
    if op == "norm_backward":
        dx, dw = s["norm"].backward(s["dy"], s["r"], s["rstd"], s["dr"]) if own else _plain_norm_backward(s)
        return {"dx": dx, "dweight": dw}
    if op == "ffn":
        return s["ffn"].forward(s["x"], s["add"]) if own else _plain_ffn(s, False)
    if op == "ffn_train":
        if not own:
            return _plain_ffn(s, True)
        out, saved = s["ffn"].forward_train(s["x"], s["add"])
        return [out] + [t for t in s["ffn"].backward(saved, s["dout"]) if t is not None]
    if not own:
        return _plain_clip(s)
    norm = s["clipper"].clip(case["max_norm"])
    return [norm] + list(s["clipped"].values())


# ---------------------------------------------------------------------------- what a pass has to do

def work(case):
    op = case["op"]
    if op in ("norm", "norm_q8"):
        T, H = case["T"], case["H"]
        b = T * H * (6 if case["residual"] else 2) + 2 * H
        if op == "norm":
            b += 2 * T * H
        else:
            b += T * H + (4 * T if case["scales"] == "row" else T * H // 32)
        return {"bytes": b, "flops": 4 * T * H}
    if op == "norm_backward":
        T, H = case["T"], case["H"]
        per = (4 if case["dy"] == "f32" else 2) + 2 + (2 if case["dr"] else 0) + 2
        return {"bytes": T * H * per + 4 * T + 6 * H, "flops": 10 * T * H}
    if op in ("ffn", "ffn_train"):
        T, H, I = case["T"], case["H"], case["I"]
        weights, rows = 2 * 3 * H * I, 2 * T * H
        b = weights + rows * (3 if case["add"] else 2) + (4 * (2 * I + H) if case["bias"] else 0)
        if op == "ffn":
            return {"bytes": b, "flops": 6 * T * H * I}
        b += weights + 2 * rows + (4 * (2 * I + H) if case["bias"] else 0)
        return {"bytes": b, "flops": 18 * T * H * I}
    n = {k: 0 for k in _TYPES}
    for name, size in _clip_shapes(case):
        n[name] += size
    return {"bytes": 2 * (4 * n["f32"] + 2 * n["bf16"] + 2 * n["f16"]) + 4, "flops": 3 * sum(n.values())}


# ---------------------------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op in ("norm", "norm_q8"):
        # the stream is kept in bf16, and what is normed is what is kept
        r = d["x"] if s["residual"] is None else (d["x"] + d["residual"]).to(torch.bfloat16).double()
        y = d["weight"] * r * torch.rsqrt(torch.einsum("th,th->t", r, r)[:, None] / case["H"] + case["eps"])
        if op == "norm":
            return {"y": y, "r": r}
        if case["scales"] == "row":
            scale = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 448.0
            scale = torch.clamp(scale, min=2.0 ** -126)
            return {"q": y / scale[:, None], "scales": scale, "r": r}
        big = torch.linalg.vector_norm(y.unflatten(1, (-1, 32)), ord=math.inf, dim=2)
        e = torch.clamp(torch.ceil(torch.log2(big / 448.0)), min=-127.0)
        return {"q": (y.unflatten(1, (-1, 32)) * torch.exp2(-e)[:, :, None]).flatten(1), "scales": None, "r": r}
    if op == "norm_backward":
        # y_h = w_h r_h / sigma: its gradient is the projection off the row's own direction
        n = d["r"] * d["rstd"][:, None]
        a = torch.einsum("th,h->th", d["dy"], d["weight"])
        dx = torch.einsum("t,th->th", d["rstd"], a - n * torch.einsum("th,th->t", a, n)[:, None] / case["H"])
        return {"dx": dx if s["dr"] is None else dx + d["dr"], "dweight": torch.einsum("th,th->h", d["dy"], n)}
    if op in ("ffn", "ffn_train"):
        I = case["I"]
        leaves = [d[k].requires_grad_(op == "ffn_train") for k in ("x", "gate_up", "down")]
        x, wgu, wdn = leaves
        g, u = torch.einsum("th,ih->ti", x, wgu[:I]), torch.einsum("th,ih->ti", x, wgu[I:])
        if case["bias"]:
            leaves += [d["gu_bias"].requires_grad_(op == "ffn_train"), d["dn_bias"].requires_grad_(op == "ffn_train")]
            g, u = g + d["gu_bias"][:I], u + d["gu_bias"][I:]
        if case["glu"]:
            g, u = g.clamp(max=GLU[1]), u.clamp(-GLU[1], GLU[1])
            h = g / (1 + torch.exp(-GLU[0] * g)) * (u + GLU[2])
        else:
            h = g / (1 + torch.exp(-g)) * u
        out = torch.einsum("ti,hi->th", h, wdn)
        if case["bias"]:
            out = out + d["dn_bias"]
        if case["add"]:
            out = out + d["add"]
        if op == "ffn":
            return out
        return [out.detach()] + list(torch.autograd.grad(out, leaves, d["dout"]))
    total = sum(float(torch.dot(f.double(), f.double())) for f in s["flat"].values()) ** 0.5
    c = min(1.0, case["max_norm"] / (total + 1e-6))
    return [total] + [f.double() * c for f in s["flat"].values()]

"""The dense operators together with the routed layer, as a block uses them (block.MoeBlock and GradClipper): a
serving step, a training step with clipping, and the same captured into a graph, against the oracles in fp64.

Tolerances are the layer's: relative Frobenius error 5e-3 for the output and 1e-2 for the gradients.  The routing is
decided on bf16 logits that both sides take from the device, since a rounding of a logit may turn a top-k choice.
The gradient of the norm's input goes through bf16 gradients of the norm's output: 1e-2 as well."""
import numpy as np
import pytest
import torch

from bit_mixture_experts_top_b200 import block, layer, synth
from bit_mixture_experts_top_b200.workloads import Workload
from helpers import bf16_to_f64, device, oracle_epilogue, oracle_lora, oracle_stacks, to_np_bits, touched_experts
from oracle import backward as obwd
from oracle import bf16, dense
from oracle import moe as omoe

pytestmark = pytest.mark.gpu

W = {
    "nf4_lora": Workload("block_nf4", "nf4", E=8, H=256, I=128, k=2, tokens=(64,), weight_std=0.05, lora_rank=8,
                         lora_alpha=16.0),
    "mxfp4_glu": Workload("block_mx", "mxfp4", E=8, H=256, I=128, k=2, tokens=(64,), exp_range=(-6, -3),
                          glu=(1.702, 7.0, 1.0), bias_std=0.2),
}


def _bits(shape, name, std=1.0):
    return synth.normal_bf16(shape, std, 0, name)


class Setup:
    def __init__(self, w, T):
        self.w, self.T = w, T
        H, I = w.H, 192
        b = dict(x=_bits((T, H), "bx"), res=_bits((T, H), "bres", 2.0), nw=_bits((H,), "bnw"),
                 rw=_bits((w.E, H), "brw", 1 / np.sqrt(H)), gu=_bits((2 * I, H), "bgu", 1 / np.sqrt(H)),
                 dn=_bits((H, I), "bdn", 1 / np.sqrt(I)), dout=_bits((T, H), "bdout"), dr=_bits((T, H), "bdr"))
        self.b = b
        self.f = {k: bf16.bf16_bits_to_f64(v) for k, v in b.items()}
        d = self.d = {k: layer.bits_tensor(v, device()) for k, v in b.items()}
        self.block = block.MoeBlock(block.RmsNorm(d["nw"], 1e-5), lambda y: y @ d["rw"].t(),
                                    layer.synthetic_layer(w, device()), block.GluFfn(d["gu"], d["dn"], glu=w.glu))

    def reference(self, train):
        w, f = self.w, self.f
        r_bits, rstd, y = dense.rmsnorm(self.b["x"], self.b["res"], self.b["nw"], 1e-5)
        y_bits = bf16.f64_to_bf16_bits(y.astype(np.float64))
        yv = bf16.bf16_bits_to_f64(y_bits)
        logits = to_np_bits(layer.bits_tensor(y_bits, device()) @ self.d["rw"].t())
        stacks = oracle_stacks(w, touched_experts(logits, w.k))
        A, B = oracle_lora(w)
        bgu, bdn = oracle_epilogue(w)
        kw = dict(lora_A_bits=A, lora_B_bits=B, lora_scale=w.lora_scale, gu_bias=bgu, dn_bias=bdn, glu=w.glu,
                  gating=w.gating)
        routed, _ = omoe.moe_forward(y_bits, logits, w.k, w.fmt, w.E, w.H, w.I, *stacks, **kw)
        out = routed + dense.ffn(yv, f["gu"], f["dn"], glu=w.glu)[0]
        if not train:
            return out, r_bits
        m = obwd.moe_backward(y_bits, logits, f["dout"], w.k, w.fmt, w.E, w.H, w.I, *stacks, **kw)
        dys, dgu, ddn, _, _ = dense.ffn_backward(yv, f["gu"], f["dn"], f["dout"], glu=w.glu)
        dx, dn = dense.rmsnorm_backward(m["dx"] + dys + m["dlogits"] @ f["rw"], bf16.bf16_bits_to_f64(r_bits), f["nw"],
                                        rstd.astype(np.float64), f["dr"])
        g = dict(dx=dx, norm=dn, gate_up=dgu, down=ddn)
        if w.lora_rank:
            g.update(lora_A=m["dA"], lora_B=m["dB"])
        return out, r_bits, g


def _rel(got, ref):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("name", sorted(W))
@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_serving_step(name, T):
    s = Setup(W[name], T)
    out, r = s.block.forward(s.d["x"], s.d["res"])
    want, r_bits = s.reference(False)
    assert np.array_equal(to_np_bits(r), r_bits)
    assert _rel(bf16_to_f64(out), want) <= 5e-3


def _step(s):
    out, r, saved = s.block.forward_train(s.d["x"], s.d["res"])
    g = s.block.backward(saved, s.d["dout"], s.d["dr"], router_grad=lambda dl: dl @ s.d["rw"].float())
    return out, r, g


@pytest.mark.parametrize("name", sorted(W))
@pytest.mark.parametrize("T", [1, 64, 300])
def test_training_step_and_clipping(name, T):
    s = Setup(W[name], T)
    out, r, g = _step(s)
    want, r_bits, ref = s.reference(True)
    assert np.array_equal(to_np_bits(r), r_bits) and _rel(bf16_to_f64(out), want) <= 5e-3
    for k, v in ref.items():
        assert _rel(g[k], v) <= 1e-2, (k, _rel(g[k], v))
    tensors = [g[k] for k in ("norm", "gate_up", "down", "lora_A", "lora_B") if g[k] is not None]
    kept = [t.double().cpu().numpy() for t in tensors]
    norm = block.GradClipper(tensors).clip(0.5)
    wn, clipped = dense.clip_grads(kept, 0.5)
    assert abs(float(norm) - wn) <= 2.0 ** -23 * wn
    for t, c in zip(tensors, clipped):
        assert _rel(t, c) <= torch.finfo(t.dtype).eps / 2 + 2.0 ** -23


def test_step_in_a_graph():
    s = Setup(W["nf4_lora"], 40)
    want_out, want_r, want = _step(s)
    want_out = want_out.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out, r, grads = _step(s)
        clipper = block.GradClipper([grads[k] for k in ("norm", "gate_up", "down", "lora_A", "lora_B")])
        norm = clipper.clip(1e9)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want_out) and torch.equal(r, want_r)
    for k in want:
        assert want[k] is None or torch.equal(grads[k], want[k]), k
    ref = np.sqrt(sum(float((want[k].double() ** 2).sum()) for k in ("norm", "gate_up", "down", "lora_A", "lora_B")))
    assert abs(float(norm) - ref) <= 2.0 ** -22 * ref


def test_refusals():
    s = Setup(W["nf4_lora"], 4)
    with pytest.raises(ValueError, match="differ in H"):
        block.MoeBlock(block.RmsNorm(s.d["nw"][:64].clone()), None, s.block.moe)
    b = block.MoeBlock(s.block.norm, lambda y: (y @ s.d["rw"].t()).float(), s.block.moe)
    with pytest.raises(ValueError, match="logits"):
        b.forward(s.d["x"])
    # without a shared expert and without a residual
    b = block.MoeBlock(s.block.norm, s.block.router, s.block.moe)
    out, r, saved = b.forward_train(s.d["x"])
    assert r.data_ptr() == s.d["x"].data_ptr()
    got = b.backward(saved, s.d["dout"])
    assert "gate_up" not in got and got["dx"].shape == (4, 256)

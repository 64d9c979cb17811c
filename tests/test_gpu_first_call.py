"""The first call of every dense operator in a process, made while a graph is captured: one-time set-up (kernel
attributes, occupancy queries) must not break the capture.  Each runs in a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
import torch
from bit_mixture_experts_top_b200 import block
what, T = sys.argv[1], int(sys.argv[2])
H, I = 512, 384
g = torch.Generator(device="cuda").manual_seed(0)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
x, w, gu, dn = r(T, H), r(H), r(2 * I, H) / 22, r(H, I) / 20
norm, ffn = block.RmsNorm(w), block.GluFfn(gu, dn)
grads = [r(1000), r(77).float()]
outs = [torch.empty_like(t) for t in grads]
clipper = block.GradClipper(grads, outs)

def step():
    if what == "norm":
        y, s, rstd = norm.forward_train(x, x)
        return [y, s, rstd, *norm.forward_q8(x, x)[:2], *norm.backward(y, s, rstd, x)]
    if what == "ffn":
        out, saved = ffn.forward_train(x, x)
        return [out, *ffn.backward(saved, x)[:3], *ffn.backward(saved, x, weights=False)[:1]]
    return [clipper.clip(0.5), *outs]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = step()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(captured, step()):
    assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))
print("same")
"""


@pytest.mark.parametrize("what,T", [("norm", 3), ("norm", 3000), ("ffn", 4), ("ffn", 30), ("ffn", 64), ("ffn", 3000),
                                    ("clip", 1)])
def test_first_call_inside_a_capture(what, T):
    r = subprocess.run([sys.executable, "-c", PROGRAM, what, str(T)], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]

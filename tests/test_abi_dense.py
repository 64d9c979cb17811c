"""CPU checks of the dense operators' entry points: argument refusals happen on the host, before anything
touches a GPU; workspace sizes; the e4b_grad layout; the checks of the block classes."""
import ctypes
import subprocess

import pytest
import torch

from bit_mixture_experts_top_b200 import block, e4b

BAD, UNSUP, OK = e4b.E4B_ERR_INVALID_ARG, e4b.E4B_ERR_UNSUPPORTED, e4b.E4B_OK
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    return e4b.lib()


def _norm(L, x=1 * MB, res=2 * MB, w=3 * MB, T=4, H=64, eps=1e-6, qf=0, r=4 * MB, y=5 * MB, q=None, qs=None, rstd=None):
    return L.e4b_rmsnorm(x, res, w, T, H, eps, qf, r, y, q, qs, rstd, None)


def test_rmsnorm_refusals(L):
    assert _norm(L, T=0) == OK                                   # no rows: nothing to do
    bad = [dict(T=-1), dict(H=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(qf=3),
           dict(x=None), dict(w=None), dict(y=None), dict(res=None),                      # r_out without a residual
           dict(q=6 * MB), dict(qf=1), dict(qf=1, q=6 * MB), dict(qf=2, qs=6 * MB),
           dict(x=MB + 1), dict(w=3 * MB + 1), dict(rstd=6 * MB + 2), dict(qf=1, q=6 * MB, qs=7 * MB + 2),
           dict(y=MB + 2), dict(y=MB - 2), dict(r=2 * MB + 64), dict(y=3 * MB), dict(y=4 * MB),   # overlaps
           dict(qf=1, q=MB, qs=7 * MB), dict(rstd=MB), dict(rstd=5 * MB + 8), dict(qf=1, q=6 * MB, qs=6 * MB)]
    for kw in bad:
        assert _norm(L, **kw) == BAD, kw
    assert _norm(L, H=40, qf=2, q=6 * MB, qs=7 * MB) == UNSUP     # MX blocks need H a multiple of 32


def _norm_bwd(L, dy=1 * MB, dt=0, dr=2 * MB, r=3 * MB, w=4 * MB, rstd=5 * MB, T=4, H=64, dx=6 * MB, dw=7 * MB,
              ws=8 * MB, n=1 << 16):
    return L.e4b_rmsnorm_backward(dy, dt, dr, r, w, rstd, T, H, dx, dw, ws, n, None)


def test_rmsnorm_backward_refusals(L):
    need = L.e4b_rmsnorm_backward_workspace_bytes(4, 64)
    assert need >= 64 * 4 and need % 256 == 0
    assert L.e4b_rmsnorm_backward_workspace_bytes(-1, 64) == 0 and L.e4b_rmsnorm_backward_workspace_bytes(4, 0) == 0
    bad = [dict(T=-1), dict(H=0), dict(dt=2), dict(dt=-1), dict(dy=None), dict(r=None), dict(w=None), dict(rstd=None),
           dict(dx=None), dict(dw=None), dict(ws=None), dict(ws=8 * MB + 8), dict(n=need - 1), dict(dy=MB + 2),
           dict(dr=2 * MB + 1), dict(rstd=5 * MB + 2), dict(dw=7 * MB + 2), dict(dx=1 * MB), dict(dx=3 * MB + 128),
           dict(dx=4 * MB), dict(dw=3 * MB), dict(dw=6 * MB), dict(ws=6 * MB), dict(dw=8 * MB)]
    for kw in bad:
        assert _norm_bwd(L, **kw) == BAD, kw


def _clip(L, items, max_norm=1.0, norm=64 * MB, ws=65 * MB, n=None, count=None):
    a = (e4b.Grad * max(1, len(items)))(*[e4b.Grad(*i, 0) for i in items])
    count = len(items) if count is None else count
    n = L.e4b_clip_grad_norm_workspace_bytes(max(0, count)) if n is None else n
    return L.e4b_clip_grad_norm(ctypes.cast(a, ctypes.c_void_p), count, max_norm, norm, ws, n, None)


def test_clip_refusals(L):
    assert L.e4b_clip_grad_norm_workspace_bytes(-1) == 0 and L.e4b_clip_grad_norm_workspace_bytes(65537) == 0
    one, many = L.e4b_clip_grad_norm_workspace_bytes(1), L.e4b_clip_grad_norm_workspace_bytes(5000)
    assert 0 < one < many and one % 256 == 0 and many % 256 == 0
    g = (MB, 2 * MB, 100, e4b.E4B_F32)
    assert _clip(L, [g], max_norm=-1.0) == BAD and _clip(L, [g], max_norm=float("nan")) == BAD
    assert _clip(L, [g], norm=None) == BAD and _clip(L, [g], norm=64 * MB + 2) == BAD
    assert _clip(L, [g], ws=None) == BAD and _clip(L, [g], ws=65 * MB + 8) == BAD and _clip(L, [g], n=one - 1) == BAD
    assert _clip(L, [g], count=-1) == BAD and _clip(L, [g], count=65537, n=1 << 30) == BAD
    assert _clip(L, [(MB, 2 * MB, 100, 3)]) == UNSUP
    for item in [(MB, 2 * MB, -1, 0), (0, 2 * MB, 4, 0), (MB, 0, 4, 0), (MB + 2, 2 * MB, 4, 0), (MB, 2 * MB + 1, 4, 1)]:
        assert _clip(L, [item]) == BAD, item
    f = e4b.E4B_F32
    overlaps = [
        [(MB, 8 * MB, 100, f), (2 * MB, 8 * MB + 396, 100, f)],         # two outs share four bytes
        [(MB, MB, 100, f), (MB, MB, 100, f)],                           # the same tensor twice in place
        [(MB, MB + 4, 100, f)],                                         # shifted onto itself
        [(MB, 8 * MB, 100, f), (8 * MB + 40, 9 * MB, 4, f)],            # an out inside another grad
        [(8 * MB, 9 * MB, 1000, f), (MB, 8 * MB + 2000, 4, f), (2 * MB, 7 * MB, 4, f)],
        [(64 * MB - 396, 9 * MB, 100, f)],                              # a grad over the norm
        [(MB, 65 * MB - 4, 100, f)],                                    # an out over the workspace
    ]
    for items in overlaps:
        assert _clip(L, items) == BAD, items
        assert _clip(L, items[::-1]) == BAD, items


def _ffn(L, d, train=False, T=32, x=MB, gu=2 * MB, dn=3 * MB, bg=4 * MB, bd=5 * MB, add=6 * MB, out=7 * MB, ws=8 * MB,
         n=16 * MB):
    call = L.e4b_ffn_forward_train if train else L.e4b_ffn_forward
    return call(ctypes.byref(d), T, x, gu, dn, bg, bd, add, out, ws, n, None)


def _ffn_bwd(L, d, T=32, x=MB, dout=2 * MB, gu=3 * MB, dn=4 * MB, dx=5 * MB, dgu=6 * MB, ddn=7 * MB, bg=8 * MB, bd=9 * MB,
             ws=10 * MB, n=16 * MB):
    return L.e4b_ffn_backward(ctypes.byref(d), T, x, dout, gu, dn, dx, dgu, ddn, bg, bd, ws, n, None)


def test_ffn_refusals(L):
    d = e4b.make_ffn_desc(64, 128)
    fw, tr = e4b.e4b_ffn_workspace_bytes(d, 32), e4b.e4b_ffn_train_workspace_bytes(d, 32)
    assert fw % 256 == 0 and fw >= 32 * 128 * 2 and tr >= fw + 32 * 256 * (4 + 2)
    for bad in [e4b.make_ffn_desc(60, 128), e4b.make_ffn_desc(64, 100), e4b.make_ffn_desc(0, 128),
                e4b.make_ffn_desc(64, -8), e4b.make_ffn_desc(64, 128, (1.702, 0.0, 1.0)),
                e4b.make_ffn_desc(64, 128, (1.702, float("nan"), 1.0)),
                e4b.make_ffn_desc(64, 128, (float("inf"), 7.0, 1.0)), e4b.FfnDesc(64, 128, 5, 0, 0, 0)]:
        assert e4b.e4b_ffn_workspace_bytes(bad, 32) == 0 and e4b.e4b_ffn_train_workspace_bytes(bad, 32) == 0
        assert _ffn(L, bad) in (BAD, UNSUP) and _ffn_bwd(L, bad) in (BAD, UNSUP)
    assert L.e4b_ffn_forward(None, 32, *[MB] * 8, MB, None) == BAD and e4b.e4b_ffn_workspace_bytes(d, -1) == 0
    bad = [dict(T=-1), dict(x=None), dict(gu=None), dict(dn=None), dict(out=None), dict(ws=None), dict(ws=8 * MB + 16),
           dict(x=MB + 8), dict(gu=2 * MB + 8), dict(dn=3 * MB + 8), dict(add=6 * MB + 8), dict(out=7 * MB + 8),
           dict(bg=4 * MB + 2), dict(bd=5 * MB + 2),
           dict(out=MB), dict(out=2 * MB), dict(out=3 * MB + 16), dict(out=5 * MB), dict(out=6 * MB + 16), dict(out=8 * MB),
           dict(x=8 * MB), dict(add=8 * MB)]
    for kw in bad:
        assert _ffn(L, d, **kw) == BAD, kw
        assert _ffn(L, d, train=True, **kw) == BAD, kw
    assert _ffn(L, d, n=fw - 1) == BAD and _ffn(L, d, train=True, n=tr - 1) == BAD
    bad = [dict(T=-1), dict(x=None), dict(dout=None), dict(gu=None), dict(dn=None), dict(ws=None), dict(n=tr - 1),
           dict(x=MB + 8), dict(dout=2 * MB + 8), dict(dx=5 * MB + 8), dict(dgu=6 * MB + 2), dict(ddn=7 * MB + 8),
           dict(bg=8 * MB + 2), dict(dx=MB), dict(dx=2 * MB), dict(dgu=3 * MB), dict(ddn=6 * MB + 16), dict(bd=8 * MB),
           dict(dx=10 * MB), dict(bg=10 * MB + 4096)]
    for kw in bad:
        assert _ffn_bwd(L, d, **kw) == BAD, kw


@pytest.mark.parametrize("cname,py", [("e4b_grad", e4b.Grad), ("e4b_ffn_desc", e4b.FfnDesc)])
def test_structs_match_the_header(tmp_path, cname, py):
    src = tmp_path / "g.c"
    fields = [f for f, _ in py._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "e4b.h"\nint main(void) {\n  printf("%zu", '
                   f"sizeof({cname}));\n" +
                   "".join(f'  printf(" %zu", offsetof({cname}, {f}));\n' for f in fields) + "  return 0;\n}\n")
    inc = e4b.HEADER.rsplit("/", 1)[0]
    subprocess.run(["gcc", "-std=c99", "-I", inc, str(src), "-o", str(tmp_path / "g")], check=True)
    got = subprocess.run([str(tmp_path / "g")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(py)] + [getattr(py, f).offset for f in fields]


def test_classes_refuse_cpu_tensors_and_wrong_shapes():
    with pytest.raises(ValueError, match="CUDA"):
        block.RmsNorm(torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match=r"\[H\]"):
        block.RmsNorm(torch.ones(4, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        block.GradClipper([torch.ones(4)])
    with pytest.raises(ValueError):
        block.GradClipper([])
    with pytest.raises(ValueError, match="CUDA"):
        block.GluFfn(torch.ones(16, 8, dtype=torch.bfloat16), torch.ones(8, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="one out per"):
        e4b.make_grads([torch.ones(4)], [])

"""The dense operators of a block around the routed 4-bit layer, on one GPU.

Thin owners of device buffers around the C ABI, as :mod:`layer` is for the
routed layer: :class:`RmsNorm` (the layer's input from the hidden stream, and
its backward), :class:`GluFfn` (the shared expert that runs next to the routed
ones, forward and backward), :class:`MoeBlock` (norm, router, routed layer and
shared expert in their order, forward and backward) and :class:`GradClipper`
(the gradients that the backward calls leave).  Nothing here computes.

Every call runs on the current stream of the tensors' device.  Outputs and
workspaces are allocated per call from torch's allocator, so calls on several
streams, and calls captured into several graphs, share nothing.

The kernels' waits are bounded.  One that runs out (a device fault or a bug: the
limit is seconds) leaves outputs that are not to be trusted; :func:`check_waits`
raises then.
"""
import contextlib
import ctypes

import torch

from . import e4b


def _check(t, name, shape, *dtypes):
    """A contiguous CUDA tensor of this shape and one of these types, or ValueError."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"e4b: {name} must be a CUDA tensor")
    if t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"e4b: {name} must be {' or '.join(str(d) for d in dtypes)} of shape {tuple(shape)}, "
                         f"got {t.dtype} of {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"e4b: {name} must be contiguous")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


_HERE = contextlib.nullcontext()


def _on(index, *tensors):
    """A context in which device ``index`` is the current one; every tensor has to be on it."""
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"e4b: a tensor on {t.device} in a call on cuda:{index}")
    return _HERE if torch._C._cuda_getDevice() == index else torch.cuda.device(index)


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _lend(stream, index, *tensors):
    """Tells the allocator that tensors saved on the raw stream `stream` are read on the current one too: dropped right
    after a backward on another stream, their memory must not be handed out on their own before that backward ends."""
    if _raw_stream(index) != stream:
        for t in tensors:
            t.record_stream(torch.cuda.current_stream(index))


def _same_desc(saved, own, what):
    if saved is not own and bytes(saved) != bytes(own):
        raise ValueError(f"e4b: the saved state is not of this {what}'s sizes and options")


def check_waits(device=None):
    """Synchronises the device's current stream and raises E4BError if a bounded wait of any call on that device, graph
    replays among them, has run out since the last check: what those calls wrote is not to be trusted."""
    with torch.cuda.device(device):
        e4b._check(e4b.e4b_wait_status(), "e4b_wait_status")


class RmsNorm:
    """Root-mean-square norm of a hidden stream [T, H] (bf16) with the residual's addition in the same pass.

    r = bf16(x + residual) (x itself without a residual), y = r * rstd * weight."""

    def __init__(self, weight: torch.Tensor, eps=1e-6):
        if weight.dim() != 1 or weight.numel() < 1:
            raise ValueError("e4b: weight must be [H]")
        self.H, self.eps = weight.numel(), float(eps)
        self.weight = _check(weight, "weight", (self.H,), torch.bfloat16)
        self.index = weight.get_device()
        self._ws_bytes = {}                     # backward workspace sizes by rows

    def _run(self, x, residual, q_format, want_rstd):
        if x.dim() != 2:
            raise ValueError("e4b: x must be [T, H]")
        T, H = x.shape[0], self.H
        _check(x, "x", (T, H), torch.bfloat16)
        if residual is not None:
            _check(residual, "residual", (T, H), torch.bfloat16)
        with _on(self.index, x, residual):
            r = x if residual is None else torch.empty_like(x)
            y = q = scales = None
            if q_format == e4b.E4B_Q8_NONE:
                y = torch.empty_like(x)
            else:
                q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
                scales = x.new_empty(T, dtype=torch.float32) if q_format == e4b.E4B_Q8_ROW else \
                    x.new_empty((T, H // 32), dtype=torch.uint8)
            rstd = x.new_empty(T, dtype=torch.float32) if want_rstd else None
            # (the tensors are checked: straight to the library, whose call costs a few microseconds in all)
            e4b._check(e4b.lib().e4b_rmsnorm(
                x.data_ptr(), _ptr(residual), self.weight.data_ptr(), T, H, self.eps, q_format,
                None if residual is None else r.data_ptr(), _ptr(y), _ptr(q), _ptr(scales), _ptr(rstd),
                e4b._stream(None)), "e4b_rmsnorm")
        return y, q, scales, r, rstd

    def forward(self, x, residual=None):
        """(y [T, H] bf16, r [T, H] bf16): the normed rows and the new stream (x itself without a residual)."""
        y, _, _, r, _ = self._run(x, residual, e4b.E4B_Q8_NONE, False)
        return y, r

    def forward_q8(self, x, residual=None, scales="mx"):
        """(q [T, H] float8_e4m3fn, scales, r): the normed rows in 8 bits.  scales "mx": E8M0 bytes [T, H / 32] (uint8),
        value = q * 2^(byte - 127); "row": fp32 [T], value = q * scale."""
        if scales not in ("mx", "row"):
            raise ValueError(f"e4b: scales must be 'mx' or 'row', got {scales!r}")
        _, q, s, r, _ = self._run(x, residual, e4b.E4B_Q8_MX if scales == "mx" else e4b.E4B_Q8_ROW, False)
        return q, s, r

    def forward_train(self, x, residual=None):
        """(y, r, rstd [T] fp32): the forward with what :meth:`backward` needs."""
        y, _, _, r, rstd = self._run(x, residual, e4b.E4B_Q8_NONE, True)
        return y, r, rstd

    def backward(self, dy, r, rstd, dr=None):
        """(dx [T, H] bf16, dweight [H] fp32) from dy [T, H] (fp32 or bf16) and, with dr [T, H] bf16, the gradient that
        reaches the stream r directly.  dx is the gradient of x and of the residual alike."""
        if r.dim() != 2:
            raise ValueError("e4b: r must be [T, H]")
        T, H = r.shape[0], self.H
        _check(r, "r", (T, H), torch.bfloat16)
        _check(rstd, "rstd", (T,), torch.float32)
        _check(dy, "dy", (T, H), torch.float32, torch.bfloat16)
        if dr is not None:
            _check(dr, "dr", (T, H), torch.bfloat16)
        with _on(self.index, dy, r, rstd, dr):
            dx = torch.empty_like(r)
            dw = r.new_empty(H, dtype=torch.float32)
            nbytes = self._ws_bytes.get(T)
            if nbytes is None:
                nbytes = self._ws_bytes[T] = e4b.e4b_rmsnorm_backward_workspace_bytes(T, H)
            ws = r.new_empty(nbytes, dtype=torch.uint8)
            e4b._check(e4b.lib().e4b_rmsnorm_backward(
                dy.data_ptr(), e4b.DTYPES[dy.dtype], _ptr(dr), r.data_ptr(), self.weight.data_ptr(), rstd.data_ptr(), T, H,
                dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), nbytes, e4b._stream(None)), "e4b_rmsnorm_backward")
        return dx, dw


class FfnSaved:
    """What :meth:`GluFfn.forward_train` keeps for :meth:`GluFfn.backward`: the input (not copied: it must not change
    before the backward) and the workspace with the pre-activations and h, whose scratch one backward at a time
    uses."""

    def __init__(self, x, ws, stream, desc):
        self.x, self.ws, self.stream, self.desc = x, ws, stream, desc


class GluFfn:
    """Gated feed-forward block with bf16 weights, the shared expert next to the routed ones:
    out = act(x W_gate^T + b, x W_up^T + b) W_down^T + b (+ add).

    gate_up [2I, H] bf16 (gate rows, then up rows), down [H, I] bf16, gu_bias [2I] / dn_bias [H] fp32 or None;
    glu = (alpha, limit, beta) selects the clamped GLU instead of SwiGLU.  H and I are multiples of 8."""

    def __init__(self, gate_up, down, gu_bias=None, dn_bias=None, glu=None):
        if down.dim() != 2:
            raise ValueError("e4b: down must be [H, I]")
        self.H, self.I = down.shape
        self.down = _check(down, "down", (self.H, self.I), torch.bfloat16)
        self.gate_up = _check(gate_up, "gate_up", (2 * self.I, self.H), torch.bfloat16)
        self.gu_bias = None if gu_bias is None else _check(gu_bias, "gu_bias", (2 * self.I,), torch.float32)
        self.dn_bias = None if dn_bias is None else _check(dn_bias, "dn_bias", (self.H,), torch.float32)
        self.index = self.down.get_device()
        self._ws_bytes = {}                     # workspace sizes by (entry point, tokens)
        with _on(self.index, self.gate_up, self.gu_bias, self.dn_bias):
            self.desc = e4b.make_ffn_desc(self.H, self.I, glu)
        if e4b.e4b_ffn_workspace_bytes(self.desc, 1) == 0:
            raise ValueError("e4b: unsupported feed-forward shape (H and I are multiples of 8, the GLU limit is "
                             "positive)")

    def _run(self, name, query, x, add, out):
        if x.dim() != 2:
            raise ValueError("e4b: x must be [T, H]")
        T = x.shape[0]
        _check(x, "x", (T, self.H), torch.bfloat16)
        if add is not None:
            _check(add, "add", (T, self.H), torch.bfloat16)
        nbytes = self._ws_bytes.get((name, T))
        if nbytes is None:
            nbytes = self._ws_bytes[name, T] = query(self.desc, T)
            if nbytes == 0:
                raise ValueError(f"e4b: {T} tokens are not supported")
        with _on(self.index, x, add, out):
            out = torch.empty_like(x) if out is None else _check(out, "out", (T, self.H), torch.bfloat16)
            ws = x.new_empty(nbytes, dtype=torch.uint8)
            e4b._check(getattr(e4b.lib(), name)(
                ctypes.byref(self.desc), T, x.data_ptr(), self.gate_up.data_ptr(), self.down.data_ptr(),
                _ptr(self.gu_bias), _ptr(self.dn_bias), _ptr(add), out.data_ptr(), ws.data_ptr(), nbytes,
                e4b._stream(None)), name)
        return out, ws

    def forward(self, x, add=None, out=None):
        """out [T, H] bf16; add [T, H] bf16 is added to it (the routed experts' output), and out may be add."""
        return self._run("e4b_ffn_forward", e4b.e4b_ffn_workspace_bytes, x, add, out)[0]

    def forward_train(self, x, add=None, out=None):
        """(out, saved): the forward, and what :meth:`backward` needs of it."""
        out, ws = self._run("e4b_ffn_forward_train", e4b.e4b_ffn_train_workspace_bytes, x, add, out)
        return out, FfnSaved(x, ws, _raw_stream(self.index), self.desc)

    def backward(self, saved, dout, weights=True):
        """(dx, d_gate_up, d_down, d_gu_bias, d_dn_bias) of sum(dout * out): bf16, the biases' fp32 (None without them).
        The gradient of add is dout.  weights False: the weights are frozen and only dx is computed, the others None."""
        _same_desc(saved.desc, self.desc, "feed-forward block")
        T = saved.x.shape[0]
        _check(dout, "dout", (T, self.H), torch.bfloat16)
        with _on(self.index, saved.x, dout):
            _lend(saved.stream, self.index, saved.x, saved.ws)
            dx = torch.empty_like(saved.x)
            dgu = torch.empty_like(self.gate_up) if weights else None
            ddn = torch.empty_like(self.down) if weights else None
            dbg = dout.new_empty(2 * self.I, dtype=torch.float32) \
                if weights and self.gu_bias is not None else None
            dbd = dout.new_empty(self.H, dtype=torch.float32) \
                if weights and self.dn_bias is not None else None
            e4b.e4b_ffn_backward(self.desc, T, saved.x, dout, self.gate_up, self.down, dx, dgu, ddn, dbg, dbd, saved.ws)
        return dx, dgu, ddn, dbg, dbd


class MoeBlock:
    """The feed-forward half of a block: norm, router, routed 4-bit layer and, where there is one, the shared expert.

    norm: :class:`RmsNorm`; moe: :class:`layer.MoeLayer`; shared: :class:`GluFfn` or None; router: a callable
    y [T, H] -> logits [T, E] (bf16), the model's own projection of the normed rows.  All parts are on one device, which
    is the current one while they, the router and its gradient run."""

    def __init__(self, norm, router, moe, shared=None):
        if moe.H != norm.H or (shared is not None and shared.H != norm.H):
            raise ValueError("e4b: the norm, the routed layer and the shared expert differ in H")
        at = {norm.index, moe.gate_up.codes.get_device(), moe.down.codes.get_device()}
        if len(at if shared is None else at | {shared.index}) != 1:
            raise ValueError("e4b: the norm, the routed layer and the shared expert are on different devices")
        self.norm, self.router, self.moe, self.shared = norm, router, moe, shared

    def _logits(self, y):
        logits = _check(self.router(y), "logits", (y.shape[0], self.moe.E), torch.bfloat16)
        _on(self.norm.index, logits)             # (the device is the current one already)
        return logits

    def forward(self, x, residual=None):
        """(out [T, H], r [T, H]): the experts' output and the stream x + residual that it is added to next."""
        with _on(self.norm.index, x, residual):
            y, r = self.norm.forward(x, residual)
            out = self.moe.forward(y, self._logits(y), ws=self.moe.new_workspace(len(y), y.device))
            return (out if self.shared is None else self.shared.forward(y, add=out, out=out)), r

    def forward_train(self, x, residual=None):
        """(out, r, saved): the forward with what :meth:`backward` needs, the routed layer's workspace among it, so other
        calls may come between a forward_train and its backward (one backward of a saved state at a time)."""
        with _on(self.norm.index, x, residual):
            y, r, rstd = self.norm.forward_train(x, residual)
            logits = self._logits(y)
            ws = self.moe.new_workspace(len(y), y.device, train=True)
            out = self.moe.forward_train(y, logits, ws=ws)
            kept = None
            if self.shared is not None:
                out, kept = self.shared.forward_train(y, add=out, out=out)
            return out, r, (y, r, rstd, logits, kept, ws, _raw_stream(self.norm.index), self.moe.desc)

    def backward(self, saved, dout, dr=None, router_grad=None, weights=True):
        """Gradients of sum(dout * out) + sum(dr * r) as a dict: dx [T, H] bf16 (of x and residual alike), norm [H]
        fp32, dlogits [T, E] fp32, lora_A / lora_B fp32 (None without LoRA) and, with a shared expert, gate_up, down,
        gu_bias and dn_bias (None where frozen or absent).  router_grad: a callable dlogits -> its part of dy [T, H],
        the router's own backward; None leaves the router's path out of dx."""
        y, r, rstd, logits, kept, ws, stream, desc = saved
        _same_desc(desc, self.moe.desc, "routed layer")
        _check(dout, "dout", y.shape, torch.bfloat16)
        with _on(self.norm.index, dout, dr):
            _lend(stream, self.norm.index, y, r, rstd, logits, ws)
            dy, dlogits, dA, dB = self.moe.backward(logits, dout, ws=ws)
            got = dict(dlogits=dlogits, lora_A=dA, lora_B=dB)
            if self.shared is not None:
                dys, *rest = self.shared.backward(kept, dout, weights)
                got.update(zip(("gate_up", "down", "gu_bias", "dn_bias"), rest))
                dy += dys
            if router_grad is not None:
                dy += router_grad(dlogits)
            got["dx"], got["norm"] = self.norm.backward(dy, r, rstd, dr)
        return got


class GradClipper:
    """Clipping of a fixed list of gradient tensors (fp32, bf16 and fp16 mixed, each contiguous) by their global norm.

    The list is described once and its tensors are held; every :meth:`clip` reads them anew.  A tensor that has been
    given other storage since (``t.data = ...``, ``set_``, a ``resize_`` that moved it) is described again; on storage
    that it keeps, a tensor has to keep its type and size too."""

    def __init__(self, grads, out=None):
        """out: tensors of the same types and sizes that take the clipped values; None clips in place."""
        self._describe(grads, out)

    def _describe(self, grads, out):
        table = e4b.make_grads(grads, out)
        grads, outs = table.tensors
        tensors = grads if outs is grads else grads + outs
        if not tensors:
            raise ValueError("e4b: no gradient tensors")
        index = tensors[0].get_device()
        with _on(index, *tensors):
            self.ws_bytes = e4b.e4b_clip_grad_norm_workspace_bytes(len(table))
            self._norm_like = tensors[0].new_empty((), dtype=torch.float32)   # (empty_like is torch's cheapest allocation)
        self.grads, self.index, self._tensors = table, index, tensors
        self._table = ctypes.addressof(table)
        # the storages are held with the addresses: nothing else can come to lie there before the next look at them
        self._storages = [t.untyped_storage() for t in tensors]
        self._addresses = list(map(torch.Tensor.data_ptr, tensors))

    def clip(self, max_norm):
        """Scales the gradients by min(1, max_norm / (norm + 1e-6)); returns the norm before clipping, a 0-d fp32
        tensor on the device.  max_norm float("inf"): the norm alone."""
        if list(map(torch.Tensor.data_ptr, self._tensors)) != self._addresses:
            grads, outs = self.grads.tensors
            self._describe(grads, None if outs is grads else outs)
        with _on(self.index):
            first = self._tensors[0]
            norm = torch.empty_like(self._norm_like)
            ws = first.new_empty(self.ws_bytes, dtype=torch.uint8)
            e4b._check(e4b.lib().e4b_clip_grad_norm(self._table, len(self.grads), float(max_norm), norm.data_ptr(), ws.data_ptr(),
                                                    self.ws_bytes, e4b._stream(None)), "e4b_clip_grad_norm")
        return norm

"""Chunkwise retention as a differentiable torch op: the forward is ret_chunkwise (or
gated_ret_chunkwise), the backward is ret_chunkwise_backward (or its gated form). Both run
in the library's kernels; this module only routes tensors. The gradients are those of the
operator from a zero initial state ("RetNet retention mechanism" page, 保留机制初识;
the Gated RetNet page's parallel_gate_retention weights for the gated form).

The operators around retention in the same manner: rotary (the prologue), msr_norm_gate (the
epilogue) and layer_norm; multi_scale_retention runs prologue, retention and epilogue. Their
gradients are not differentiable again: a second backward raises.

Capturing a backward in a CUDA graph: take the gradients with torch.autograd.grad, and let go of
eager graphs over the same leaves first. backward() accumulates into the leaves on the stream on
which an earlier graph met them, which a capture on another stream cannot wait for."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import ret


class ChunkwiseRetention(torch.autograd.Function):
    """o = retention(q, k, v; decay). decay: gamma [H] (gated=False) or g [B, H, N] (gated=True)."""

    @staticmethod
    def forward(ctx, q, k, v, decay, chunk: int, gated: bool):
        q, k, v, decay = (t.contiguous() for t in (q, k, v, decay))
        if gated:
            o = ret.gated_ret_chunkwise(q, k, v, decay, chunk)
        else:
            o = ret.ret_chunkwise(q, k, v, decay, chunk)
        ctx.save_for_backward(q, k, v, decay)
        ctx.chunk, ctx.gated = chunk, gated
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, decay = ctx.saved_tensors
        want_decay = ctx.needs_input_grad[3]
        dq, dk, dv, dd = ret.chunkwise_backward(q, k, v, decay, do.contiguous(), ctx.chunk, gated=ctx.gated,
                                                ddecay=want_decay)
        return dq, dk, dv, dd, None, None


def chunkwise_retention(q, k, v, decay, chunk: int = 64, gated: bool = False):
    """Differentiable chunkwise retention (see ChunkwiseRetention); o has v's layout and q's dtype."""
    return ChunkwiseRetention.apply(q, k, v, decay, chunk, gated)


class Rotary(torch.autograd.Function):
    """(q_out, k_out) = ret.rotary(q, k, ...); k may be None."""

    @staticmethod
    def forward(ctx, q, k, freqs, positions, starts, kwargs):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(freqs, positions, starts)
        ctx.kwargs = kwargs
        return ret.rotary(q, k, freqs, positions=positions, starts=starts, **kwargs)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        freqs, positions, starts = ctx.saved_tensors
        kw = dict(positions=positions, starts=starts, **ctx.kwargs)
        if dq is None and dk is None:
            return (None,) * 6
        dq, dk = (None if t is None else t if t.stride(-1) == 1 else t.contiguous() for t in (dq, dk))
        if dq is None:  # the gradient reaches k alone: its turn in q's place
            kw["q_scale"] = kw["k_scale"]
            return None, ret.rotary_backward(dk, None, freqs, **kw)[0], None, None, None, None
        return (*ret.rotary_backward(dq, dk, freqs, **kw), None, None, None, None)


def rotary(q, k, freqs, positions=None, starts=None, offset=0, layout="interleaved", amplitude=1.0, q_scale=1.0,
           k_scale=1.0):
    """Differentiable ret.rotary: token-major q, k [B, N, H, d] to rotated head-major [B, H, N, d] (k may be None)."""
    return Rotary.apply(q, k, freqs, positions, starts, dict(offset=offset, layout=layout, amplitude=amplitude,
                                                             q_scale=q_scale, k_scale=k_scale))


class MsrNormGate(torch.autograd.Function):
    """y = ret.msr_norm_gate(o, gate, eps)."""

    @staticmethod
    def forward(ctx, o, gate, eps: float):
        o, gate = o.contiguous(), gate.contiguous()
        ctx.save_for_backward(o, gate)
        ctx.eps = eps
        return ret.msr_norm_gate(o, gate, eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        o, gate = ctx.saved_tensors
        return (*ret.msr_norm_gate_backward(dy.contiguous(), o, gate, ctx.eps), None)


def msr_norm_gate(o, gate, eps: float = 1e-5):
    """Differentiable ret.msr_norm_gate: o [B, H, N, dv], gate [B, N, H, dv], y [B, N, H, dv]. The kernel takes
    contiguous tensors: a gate that is a slice of a fused projection is copied first, and the copy kept for the
    backward."""
    return MsrNormGate.apply(o, gate, eps)


class LayerNorm(torch.autograd.Function):
    """(y, s) of ret.layer_norm; s is None without a residual."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps: float, residual):
        ctx.set_materialize_grads(False)
        x, weight, bias, residual = (None if t is None else t.contiguous() for t in (x, weight, bias, residual))
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        out = ret.layer_norm(x, weight, bias, eps, residual=residual, mean=mean, rstd=rstd)
        y, s = (out, None) if residual is None else out
        ctx.save_for_backward(x if s is None else s, weight, mean, rstd)
        ctx.wdtype = None if bias is None else bias.dtype
        return y, s

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum):
        x, weight, mean, rstd = ctx.saved_tensors
        if dy is None:  # only the sum was used: its gradient passes through
            return dsum, None, None, None, dsum if ctx.needs_input_grad[4] else None
        dx, dw, db = ret.layer_norm_backward(dy.contiguous(), x, weight, mean, rstd,
                                             dsum=None if dsum is None else dsum.contiguous(),
                                             dweight=ctx.needs_input_grad[1], dbias=ctx.needs_input_grad[2],
                                             wdtype=ctx.wdtype)
        return dx, dw, db, None, dx if ctx.needs_input_grad[4] else None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, residual=None):
    """Differentiable ret.layer_norm: y, or (y, x + residual) with a residual."""
    y, s = LayerNorm.apply(x, weight, bias, eps, residual)
    return y if residual is None else (y, s)


def multi_scale_retention(q, k, v, gate, decay, freqs=None, chunk: int = 64, gated: bool = False, eps: float = 1e-5,
                          positions=None, starts=None, offset=0, layout="interleaved", amplitude=1.0, q_scale=1.0,
                          k_scale=1.0):
    """RetNet's multi-scale retention between its projections, differentiable: q, k [B, N, H, dk], v and gate
    [B, N, H, dv] token-major (slices of a fused projection too; q, k and v are read in place, such a gate is copied),
    decay gamma [H] or g [B, H, N]; returns [B, N, H, dv] for the output projection. Rotary prologue, chunkwise
    retention, norm and gate."""
    qh, kh = rotary(q, k, freqs, positions, starts, offset, layout, amplitude, q_scale, k_scale)
    vh, _ = rotary(v, None, None)  # layout only
    return msr_norm_gate(chunkwise_retention(qh, kh, vh, decay, chunk, gated), gate, eps)

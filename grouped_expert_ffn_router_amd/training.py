"""The block's operators under torch's autograd: each a forward call of ``block`` whose backward pass is that module's.

Gradients are once differentiable.  A step that is captured into a HIP graph calls ``block``'s functions themselves: autograd
ties a leaf's gradient to the stream of the graph that was built first.
"""

import torch
from torch.autograd.function import once_differentiable

from . import block


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        y, s = block.rms_norm(x, weight, residual=residual, eps=eps)
        ctx.save_for_backward(s, weight)
        ctx.eps, ctx.added = eps, residual is not None
        return (y, s) if ctx.added else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, weight = ctx.saved_tensors
        if dy is None:   # only the sum was used
            return ds, None, ds, None
        dx, dweight = block.rms_norm_backward(dy.contiguous(), s, weight, dstream=None if ds is None else ds.contiguous(),
                                              eps=ctx.eps)
        return dx, dweight.to(weight.dtype), dx if ctx.added else None, None


class _Select(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, rule):
        idx, w = block.select_experts(logits, rule)
        ctx.save_for_backward(logits, idx, w)
        ctx.rule = rule
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dw):
        logits, idx, w = ctx.saved_tensors
        return block.select_experts_backward(dw, w, idx, logits, ctx.rule), None


class _Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate_up, counts):
        h, saved = block.swiglu_checkpoint(gate_up, counts)
        ctx.save_for_backward(saved.codes, saved.scales, counts)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        codes, scales, counts = ctx.saved_tensors
        saved = block.Mx8Rows(codes, scales, codes.shape[-1])
        return block.swiglu_backward(dh.contiguous(), saved, counts, hidden=False)[0], None


def rms_norm(x, weight, residual=None, eps=1e-6):
    """block.rms_norm with gradients: (y, x + residual), or y alone without a residual."""
    return _Norm.apply(x, weight, residual, eps)


def select_experts(logits, rule):
    """block.select_experts with the weights' gradient to the logits: (idx, w)."""
    return _Select.apply(logits, rule)


def swiglu(gate_up, counts=None):
    """block.swiglu_checkpoint's h; what the graph keeps for the backward pass are gate_up's MX-FP8 rows in its place."""
    return _Swiglu.apply(gate_up, counts)

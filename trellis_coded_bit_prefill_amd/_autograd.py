"""What torch's autograd records for adapters(), gated(), cross_entropy(),
distill() and embed(): the calls themselves, and their backward passes
adapters_backward(), gated_backward(), loss_backward() and embed_backward() as
the gradients. Loaded by the first call that a graph is recorded for.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

import trellis_coded_bit_prefill_amd as tp


def refuse_capture(what):
    """A recorded call and its backward pass stay out of captures: there the
    leaves' gradients are added up on the streams of whichever graphs of them
    live, and a stream outside the capture that takes part ends the capture or
    the process. The calls themselves can be captured under torch.no_grad()."""
    if torch.cuda.is_current_stream_capturing():
        gradients = "keep=True and loss_backward()" if what in ("cross_entropy", "distill") else f"{what}_backward()"
        raise ValueError(f"{what}() is not differentiated while its stream is captured: capture it under "
                         f"torch.no_grad(), with {gradients} for the gradients")


def _rows(grad):
    """A gradient as the library takes it: autograd hands over expanded ones and
    slices of larger ones."""
    grad = grad.contiguous()
    return grad.clone() if grad.data_ptr() % 16 else grad


class Adapters(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, codes, scales, bits, a, b, gain, index):
        ctx.bits = bits
        ctx.save_for_backward(x, codes, scales, a, b, gain, index)
        return tp.adapters(x, codes, scales, bits, a, b, gain, index)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        refuse_capture("adapters")
        x, codes, scales, a, b, gain, index = ctx.saved_tensors
        dx, da, db = tp.adapters_backward(_rows(dout), x, codes, scales, ctx.bits, a, b, gain, index)
        need = ctx.needs_input_grad
        return dx if need[0] else None, None, None, None, da if need[4] else None, db if need[5] else None, None, None


class Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, codes_gate, scales_gate, codes_up, scales_up, bits, keep):
        h, gate, up = tp.gated(x, codes_gate, scales_gate, codes_up, scales_up, bits, keep=True)
        ctx.bits = bits
        ctx.save_for_backward(gate, up, codes_gate, scales_gate, codes_up, scales_up)
        ctx.set_materialize_grads(False)
        return (h, gate, up) if keep else h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dgate=None, dup=None):
        refuse_capture("gated")
        if dgate is not None or dup is not None:
            raise RuntimeError("gated(): the kept projections are what gated_backward() takes; a gradient of their "
                               "own is not carried back to x")
        if dh is None:
            return (None,) * 7
        dx = tp.gated_backward(_rows(dh), *ctx.saved_tensors, ctx.bits)[0]
        return (dx,) + (None,) * 6


def _loss_outputs(ctx, out, keep):
    """loss, lse[, dx]: dx is kept for the backward pass, and loss alone is differentiated."""
    loss, lse, dx = out
    ctx.save_for_backward(dx)
    ctx.set_materialize_grads(False)
    if keep:
        dx = dx.view_as(dx)
        ctx.mark_non_differentiable(dx)
        return loss, lse, dx
    return loss, lse


def _loss_gradient(ctx, what, dloss, dlse):
    refuse_capture(what)
    if dlse is not None:
        raise RuntimeError(f"{what}(): a gradient of lse is not carried back to x")
    if dloss is None:
        return None
    dx, = ctx.saved_tensors
    return tp.loss_backward(dloss.contiguous(), dx)


class CrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, codes, scales, bits, target, keep):
        return _loss_outputs(ctx, tp.cross_entropy(x, codes, scales, bits, target, keep=True), keep)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, dlse, *_):
        return (_loss_gradient(ctx, "cross_entropy", dloss, dlse),) + (None,) * 5


class Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, codes, scales, bits, index, logits, temperature, keep):
        return _loss_outputs(ctx, tp.distill(x, codes, scales, bits, index, logits, temperature, keep=True), keep)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, dlse, *_):
        return (_loss_gradient(ctx, "distill", dloss, dlse),) + (None,) * 7


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, codes, scales, k, bits, scale, extra):
        ctx.save_for_backward(tokens)
        ctx.at = codes.shape[0], extra.shape[0], scale
        return tp.embed(tokens, codes, scales, k, bits, scale, extra)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        refuse_capture("embed")
        tokens, = ctx.saved_tensors
        if ctx.at[1] == 0:  # (no trained rows: embed_backward() takes one at least)
            return (None,) * 6 + (dout.new_empty((0, dout.shape[1])),)
        return (None,) * 6 + (tp.embed_backward(_rows(dout), tokens, *ctx.at),)

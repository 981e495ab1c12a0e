"""What torch's autograd records for adapters() and gated(): the calls
themselves, and their backward passes adapters_backward() and
gated_backward() as the gradients. Loaded by the first call that a graph is
recorded for.
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
        raise ValueError(f"{what}() is not differentiated while its stream is captured: capture it under "
                         f"torch.no_grad(), with {what}_backward() for the gradients")


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

"""Differentiable solve x = A^-1 b as a torch.autograd.Function.

Forward runs the library's PCG (M^-1 = G G^T + eps I); backward runs the
library's adjoint solve A^T lambda = dL/dx and returns dL/db = lambda and
dL/dvals[k] = -lambda_row(k) x_col(k) on A's stored entries ("torch-sla",
Technical Summary, Methodology 2: one adjoint solve, gradient only on the
sparsity pattern, O(n + nnz) memory independent of the iteration count).
Only x is saved between forward and backward.

linear_recurrence does the same for the lower bidiagonal system of a gated
recurrence along a sequence: forward substitution, and the transposed solve
for the gradients; besides the inputs it saves a state every 128 steps.

The gradients are differentiable no further: differentiating them raises.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as B


class PCGSolve(torch.autograd.Function):
    @staticmethod
    def forward(ctx, vals, b, A: B.Mat, G: B.Mat, eps: float, rtol: float, maxit: int):
        # `vals` must be the tensor A was created from (the handle borrows it).
        if vals.data_ptr() != A._keep[2].data_ptr():
            raise ValueError("vals must be the value tensor the handle A borrows")
        x, info = B.sla_pcg_solve(A, G, eps, b.contiguous(), rtol=rtol, maxit=maxit)
        ctx.save_for_backward(x)
        ctx.A, ctx.G, ctx.eps, ctx.rtol, ctx.maxit = A, G, eps, rtol, maxit
        ctx.info = info
        return x

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_x):
        (x,) = ctx.saved_tensors
        grad_b, grad_vals, _ = B.sla_pcg_adjoint(ctx.A, ctx.G, ctx.eps, x, grad_x.contiguous(),
                                                 rtol=ctx.rtol, maxit=ctx.maxit)
        return grad_vals, grad_b, None, None, None, None, None


def solve(vals, b, A: B.Mat, G: B.Mat, eps: float = 3e-3, rtol: float = 1e-10,
          maxit: int = 5000):
    """x = A^-1 b, differentiable in A's stored values and in b."""
    return PCGSolve.apply(vals, b, A, G, eps, rtol, maxit)


class LinearRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, h0, offsets, mode):
        h, last, saved = B.sla_linrec_forward(x, gate, h0=h0, offsets=offsets, mode=mode,
                                              save=any(ctx.needs_input_grad))
        ctx.save_for_backward(x, gate, h0, offsets, saved)
        ctx.mode = mode
        ctx.set_materialize_grads(False)
        return h, last

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_h, grad_last):
        x, gate, h0, offsets, saved = ctx.saved_tensors
        if grad_h is not None and grad_h.shape[-1] > 1 and grad_h.stride(-1) != 1:
            grad_h = grad_h.contiguous()  # e.g. the expanded gradient of a sum
        if grad_last is not None:
            grad_last = grad_last.contiguous()
        dx, dgate, dh0 = B.sla_linrec_backward(x, gate, saved, grad_h, grad_last=grad_last, h0=h0,
                                               offsets=offsets, mode=ctx.mode)
        return dx, dgate, dh0, None, None


def linear_recurrence(x, gate, h0=None, offsets=None, mode: str = "sigmoid"):
    """(h, last states) of the recurrence that binding.sla_linrec_forward
    describes, differentiable in x, gate and h0."""
    return LinearRecurrence.apply(x, gate, h0, offsets, mode)

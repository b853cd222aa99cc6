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

causal_conv, selective_scan, norm_in and norm_out wrap the operators of a
sequence block and their adjoints in the same manner.

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


def _rows(grad):
    """A gradient whose channels are adjacent (that of a sum is expanded)."""
    if grad is not None and grad.shape[-1] > 1 and grad.stride(-1) != 1:
        return grad.contiguous()
    return grad


def _dense(grad):
    return None if grad is None else grad.contiguous()


class CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, state, offsets, act):
        ctx.save_for_backward(x, weight, bias, state, offsets)
        ctx.act = act
        ctx.set_materialize_grads(False)
        return B.sla_conv_forward(x, weight, bias=bias, state=state, offsets=offsets, act=act)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_last):
        x, weight, bias, state, offsets = ctx.saved_tensors
        grads = B.sla_conv_backward(x, weight, _rows(grad_y), bias=bias, state=state,
                                    grad_last=_dense(grad_last), offsets=offsets, act=ctx.act)
        return (*grads, None, None)


def causal_conv(x, weight, bias=None, state=None, offsets=None, act: str = "silu"):
    """(y, last inputs) of the convolution that binding.sla_conv_forward describes,
    differentiable in x, weight, bias and state."""
    return CausalConv.apply(x, weight, bias, state, offsets, act)


class SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, Bs, Cs, D, z, dt_bias, h0, offsets, softplus):
        y, last, saved = B.sla_selscan_forward(x, dt, A, Bs, Cs, D=D, z=z, dt_bias=dt_bias, h0=h0,
                                               offsets=offsets, softplus=softplus,
                                               save=any(ctx.needs_input_grad))
        ctx.save_for_backward(x, dt, A, Bs, Cs, D, z, dt_bias, h0, offsets, saved)
        ctx.softplus = softplus
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_last):
        x, dt, A, Bs, Cs, D, z, dt_bias, h0, offsets, saved = ctx.saved_tensors
        grad_y = torch.zeros_like(x) if grad_y is None else _rows(grad_y)
        grads = B.sla_selscan_backward(x, dt, A, Bs, Cs, saved, grad_y,
                                       grad_last=_dense(grad_last), D=D, z=z, dt_bias=dt_bias,
                                       h0=h0, offsets=offsets, softplus=ctx.softplus)
        return (*grads, None, None)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, offsets=None,
                   softplus: bool = True):
    """(y, last states) of the scan that binding.sla_selscan_forward describes,
    differentiable in all tensors but the offsets; besides them it saves a state every
    16 steps (8 in float64) if any of them requires a gradient, under torch.no_grad too:
    binding.sla_selscan_forward keeps none unless asked, and takes few steps faster so."""
    return SelectiveScan.apply(x, dt, A, B, C, D, z, dt_bias, h0, offsets, softplus)


class NormIn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, scale, eps):
        y, r, rstd = B.sla_norm_in_forward(x, weight, residual=residual, scale=scale, eps=eps)
        ctx.save_for_backward(x, weight, residual, scale, rstd)
        ctx.set_materialize_grads(False)
        return y, None if r is x else r

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_r):
        x, weight, residual, scale, rstd = ctx.saved_tensors
        grad_y = torch.zeros_like(x, memory_format=torch.contiguous_format) if grad_y is None \
            else grad_y.contiguous()
        dx, dres, dw, dscale = B.sla_norm_in_backward(grad_y, x, weight, rstd, residual=residual,
                                                      scale=scale, grad_r=_dense(grad_r))
        return dx, dw, dres if residual is not None else None, dscale, None


def norm_in(x, weight, residual=None, scale=None, eps: float = 1e-5):
    """(y, r) of the norm before a block that binding.sla_norm_in_forward describes,
    differentiable in x, weight, residual and scale; without the last two r is x."""
    y, r = NormIn.apply(x, weight, residual, scale, eps)
    return y, x if r is None else r


class NormOut(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, gate, residual, scale, order, eps):
        out, rstd = B.sla_norm_out_forward(x, weight, gate=gate, residual=residual, scale=scale,
                                           order=order, eps=eps)
        ctx.save_for_backward(x, weight, gate, scale, rstd)
        ctx.order, ctx.added = order, residual is not None
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, weight, gate, scale, rstd = ctx.saved_tensors
        grad_out = grad_out.contiguous()
        dx, dgate, dw, dscale = B.sla_norm_out_backward(grad_out, x, weight, rstd, gate=gate,
                                                        scale=scale, order=ctx.order)
        return dx, dw, dgate, grad_out if ctx.added else None, dscale, None, None


def norm_out(x, weight, gate=None, residual=None, scale=None, order: str = "gate_first",
             eps: float = 1e-5):
    """The gated norm after a block that binding.sla_norm_out_forward describes,
    differentiable in all tensors."""
    return NormOut.apply(x, weight, gate, residual, scale, order, eps)

"""The autograd functions with plain stand-ins for the library's calls (no GPU):
first-order gradients come out, and differentiating them again raises instead of
dropping what the solves contribute."""
import pytest
import torch

from preconditioned_cg_solver_amd import autograd as AG
from preconditioned_cg_solver_amd import binding as B
from preconditioned_cg_solver_amd import studies


def forward(x, gate, h0=None, offsets=None, mode="sigmoid", save=False):
    h, hs = (torch.zeros_like(x[:, 0]) if h0 is None else h0), []
    for t in range(x.shape[1]):
        h = gate[:, t] * h + x[:, t]
        hs.append(h)
    return torch.stack(hs, 1), h, torch.zeros(1) if save else None


def backward(x, gate, saved, grad_h, grad_last=None, h0=None, offsets=None, mode="sigmoid"):
    h, _, _ = forward(x, gate, h0)
    mu = torch.zeros_like(x[:, 0]) if grad_last is None else grad_last
    dx, dg = torch.zeros_like(x), torch.zeros_like(x)
    for t in reversed(range(x.shape[1])):
        lam = mu if grad_h is None else grad_h[:, t] + mu
        dx[:, t] = lam
        dg[:, t] = lam * (h[:, t - 1] if t else h0)
        mu = gate[:, t] * lam
    return dx, dg, mu


class Handle:
    def __init__(self, a, vals=None):
        self.a, self._keep = a, (None, None, vals)


def twice(loss, inputs):
    grads = torch.autograd.grad(loss, inputs, create_graph=True)
    penalty = loss + sum(g.square().sum() for g in grads)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        penalty.backward()
    return grads


def test_recurrence(monkeypatch):
    monkeypatch.setattr(B, "sla_linrec_forward", forward)
    monkeypatch.setattr(B, "sla_linrec_backward", backward)
    gen = torch.Generator().manual_seed(1)
    args = [torch.rand(s, generator=gen, dtype=torch.float64).requires_grad_()
            for s in ((2, 4, 3), (2, 4, 3), (2, 3))]
    assert torch.autograd.gradcheck(
        lambda x, g, h0: AG.linear_recurrence(x, g, h0, mode="linear"), args)
    h, last = AG.linear_recurrence(*args, mode="linear")
    twice(h.square().sum() + last.sum(), args)


def test_solve(monkeypatch):
    a = torch.tensor([2.0, 3.0, 4.0], dtype=torch.float64, requires_grad=True)  # diagonal
    b = torch.ones(3, dtype=torch.float64, requires_grad=True)
    monkeypatch.setattr(B, "sla_pcg_solve", lambda A, G, eps, b, **kw: (b / A.a.detach(), None))
    monkeypatch.setattr(B, "sla_pcg_adjoint", lambda A, G, eps, x, g, **kw:
                        (g / A.a.detach(), -g / A.a.detach() * x, None))
    x = AG.solve(a, b, Handle(a, a), None)
    grads = twice(x.square().sum(), [a, b])
    assert torch.allclose(grads[1], 2 * x / a) and torch.allclose(grads[0], -2 * x * x / a)


def test_solve_of_columns(monkeypatch):
    a = torch.tensor([[2.0], [4.0]], dtype=torch.float64)
    monkeypatch.setattr(B, "sla_pcg_solve_multi", lambda A, G, eps, b, **kw: (b / A.a, None))
    monkeypatch.setattr(B, "sla_pcg_adjoint_multi", lambda A, G, eps, x, g, **kw: (g / A.a, None))
    rhs = torch.ones(2, 3, dtype=torch.float64, requires_grad=True)
    x = studies._SolveColumns.apply(rhs, Handle(a), None, 3e-3, 1e-10, 10)
    (grad,) = twice(x.square().sum(), [rhs])
    assert torch.allclose(grad, 2 * x / a)

"""Studies run through the library's kernels (reports, not the hot path).

* ``jacobi``: PCG with the factorised SPAI preconditioner (seeded random G on
  A's lower pattern, eps = 3e-3) against diagonal (Jacobi) preconditioning,
  M^-1 = D^-1 (G = diag(a_ii^-1/2), eps = 0), through the same kernels; and
  an eps sweep (3e-5 ... 3e-1) of the SPAI preconditioner.  This mirrors the
  learned-SPAI page's "Measured effects" table (Diagonal vs SPAI total solve
  time; the eps ablation) on the synthetic workloads -- with a random G,
  not the learned one, so the iteration counts are not the pages'.

* ``quality``: the preconditioner-quality metrics of the learned-SPAI page's
  setup for the same two preconditioners: the condition number of M^-1 A
  estimated from the solve's own CG coefficients (extreme eigenvalues of the
  Lanczos tridiagonal) and the scale-invariant SAI loss
  || A M^-1 / s - I ||_F^2 / n estimated with Rademacher probes, s being the
  mean absolute stored entry of A.

* ``trace``: one forward and one adjoint solve (with dL/dA) of a power-law
  SPD system of ``--rows`` rows (default 20,000) on its locality ordering:
  the run to record with ``SLA_TRACE=1`` under ``rocprofv3 --marker-trace``,
  which shows the library's phases (handle creation, the ordering, the
  solves, the pattern gradient) around their kernels.

* ``learn``: coefficients of a model learnt through the solver (the inverse
  problem of "torch-sla", applications: an optimiser's loop through the
  solve).  Sources on the nodes of a 64 x 64 grid relax towards a driving
  signal, h_t = a h_{t-1} + (1 - a) s u_t with a rate a = sigmoid(g) and a
  strength s per node; some of the fields that they cause over a short time
  by diffusion, A x_t = h_t with A = I + dt L / h^2, are observed.  g and s
  are learnt from the observations: the recurrence along time
  (autograd.linear_recurrence), the solves of all observed times at once,
  their adjoint, the recurrence's adjoint and an AdamW step over both
  parameters, with states of ``--bits`` bits.

Usage: ``python -m preconditioned_cg_solver_amd.studies
jacobi|quality|trace|learn [--configs 0,1,2,3] [--rows N] [--iters N]
[--bits 8|32]``.  jacobi and quality print one JSON line per configuration,
learn one for the run.
"""
from __future__ import annotations

import argparse
import json
import time

import numpy as np
import torch
from torch.autograd.function import once_differentiable

from . import autograd as AG
from . import binding as B
from . import inputs as I


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def _handle(M, transpose=False):
    arrs = (_dev(M.row_ptr), _dev(M.col_idx), _dev(M.vals))
    if M.block_dim == 1:
        return B.sla_csr_create(*arrs, build_transpose=transpose)
    return B.sla_bsr_create(*arrs, block_dim=M.block_dim, build_transpose=transpose)


def _timed_solve(A, G, eps, b, rtol, maxit, work, reps=3):
    x = torch.empty_like(b)
    B.sla_pcg_solve(A, G, eps, b, x=x, rtol=rtol, maxit=maxit, work=work)
    ts, info = [], None
    for _ in range(reps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        _, info = B.sla_pcg_solve(A, G, eps, b, x=x, rtol=rtol, maxit=maxit, work=work)
        ts.append(time.perf_counter() - t0)
    return info, float(np.median(ts))


def jacobi(configs):
    for c in configs:
        p = I.make_problem(c)
        A = _handle(p.A)
        G = _handle(p.G, transpose=True)
        D = _handle(I.diagonal_factor(p.A), transpose=True)
        b = _dev(p.b)
        work = B.workspace(A)
        spai, t_spai = _timed_solve(A, G, p.eps, b, p.rtol, p.maxit, work)
        diag, t_diag = _timed_solve(A, D, 0.0, b, p.rtol, p.maxit, work)
        sweep = {}
        for eps in (3e-5, 3e-4, 3e-3, 3e-2, 3e-1):
            info, t = _timed_solve(A, G, eps, b, p.rtol, p.maxit, work, reps=1)
            sweep[f"{eps:g}"] = {"iterations": info.iterations, "ms": round(t * 1e3, 2),
                                 "status": B.sla_status_string(info.status)}
        print(json.dumps({
            "config": p.name, "n": p.A.n, "nnz": p.A.nnz, "rtol": p.rtol,
            "spai": {"eps": p.eps, "iterations": spai.iterations, "ms": round(t_spai * 1e3, 2)},
            "jacobi": {"iterations": diag.iterations, "ms": round(t_diag * 1e3, 2)},
            "eps_sweep": sweep}), flush=True)
        for h in (A, G, D):
            h.destroy()


def _quality(A, G, eps, b, rtol, maxit, probes, scale):
    _, info, al, be = B.sla_pcg_solve_history(A, G, eps, b, rtol=rtol, maxit=maxit,
                                              raise_on_error=False)
    lo, hi = B.sla_lanczos_extremes(al.numpy(), be.numpy())
    loss = B.sla_sai_loss(A, G, eps, probes, scale)
    n = probes.shape[0]
    return {"iterations": info.iterations, "ritz_min": lo, "ritz_max": hi, "kappa_est": hi / lo,
            "sai_loss_per_n": float(loss.mean().item()) / n}


def quality(configs, nprobe=16):
    for c in configs:
        p = I.make_problem(c)
        A = _handle(p.A)
        G = _handle(p.G, transpose=True)
        D = _handle(I.diagonal_factor(p.A), transpose=True)
        b = _dev(p.b)
        W = np.random.default_rng(1000 + c).choice([-1.0, 1.0], size=(p.A.n, nprobe))
        probes = _dev(W)
        scale = float(np.mean(np.abs(p.A.vals)))
        print(json.dumps({
            "config": p.name, "n": p.A.n, "rtol": p.rtol, "probes": nprobe, "scale": scale,
            "spai": dict(eps=p.eps, **_quality(A, G, p.eps, b, p.rtol, p.maxit, probes, scale)),
            "jacobi": _quality(A, D, 0.0, b, p.rtol, p.maxit, probes, scale)}), flush=True)
        for h in (A, G, D):
            h.destroy()


def trace_run(rows: int):
    """One forward and one adjoint solve of a seeded power-law SPD system
    (16 random neighbours per row, Zipf 2.1 column weights, factorised SPAI
    eps = 3e-3), forced onto its locality ordering."""
    import os
    os.environ.setdefault("SLA_ORDER", "1")
    rng = np.random.default_rng([20, rows])
    A = I.powerlaw_spd(rows, rng)
    G = I.spai_factor(A, rng)
    b = rng.standard_normal(rows)
    dev = torch.device("cuda:0")

    def mk(M, transpose=False):
        return B.sla_csr_create(torch.as_tensor(M.row_ptr.astype(np.int32), device=dev),
                                torch.as_tensor(M.col_idx.astype(np.int32), device=dev),
                                torch.as_tensor(M.vals, device=dev), build_transpose=transpose)
    Ah, Gh = mk(A), mk(G, transpose=True)
    bt = torch.as_tensor(b, device=dev)
    x, info = B.sla_pcg_solve(Ah, Gh, 3e-3, bt, rtol=1e-8, maxit=2000)
    _, _, ainfo = B.sla_pcg_adjoint(Ah, Gh, 3e-3, x, bt, rtol=1e-8, maxit=2000)
    print(json.dumps({"rows": rows, "nnz": int(A.nnz), "reordered": B.sla_mat_reordered(Ah),
                      "iterations": info.iterations, "adjoint_iterations": ainfo.iterations}),
          flush=True)


class _SolveColumns(torch.autograd.Function):
    """X = A^-1 B for the columns of B, with the adjoint solves as its gradient."""

    @staticmethod
    def forward(ctx, rhs, A, G, eps, rtol, maxit):
        ctx.args = (A, G, eps, rtol, maxit)
        return B.sla_pcg_solve_multi(A, G, eps, rhs.contiguous(), rtol=rtol, maxit=maxit)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        A, G, eps, rtol, maxit = ctx.args
        # A does not depend on the parameters: of its adjoint only dL/dB is used
        x = torch.zeros_like(grad)
        out = B.sla_pcg_adjoint_multi(A, G, eps, x, grad.contiguous(), rtol=rtol, maxit=maxit)
        return out[0], None, None, None, None, None


def learn(iters: int = 300, bits: int = 32, steps: int = 256, snapshots: int = 16, lr: float = 0.05,
          seed: int = 0):
    """Learn relaxation rates and source strengths from observed fields."""
    rng = np.random.default_rng([21, seed])
    M = I.heat2d(64, dt=1e-4)
    A, G = _handle(M), _handle(I.spai_factor(M, rng), transpose=True)
    n = M.n
    drive = _dev(np.cumsum(rng.standard_normal(steps)) / 4.0)
    seen = _dev(np.linspace(steps // 8, steps - 1, snapshots).astype(np.int64))
    true_g = _dev(3.0 + 0.5 * rng.standard_normal(n))
    true_s = _dev(1.0 + 0.3 * rng.standard_normal(n))

    def fields(g, s):
        x = drive[None, :, None] * s
        h, _ = AG.linear_recurrence(x, g.expand(1, steps, n))
        return _SolveColumns.apply(h[0, seen].t(), A, G, 3e-3, 1e-10, 500)

    with torch.no_grad():
        observed = fields(true_g, true_s)
    scale = float(observed.square().mean())
    g = torch.full_like(true_g, 3.0, requires_grad=True)
    s = torch.ones_like(true_s, requires_grad=True)
    opt = B.sla_adamw_create([g, s], state_bits=bits)
    losses, t0 = [], None
    for t in range(1, iters + 1):
        if t == 2:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        loss = (fields(g, s) - observed).square().mean() / scale
        grads = torch.autograd.grad(loss, [g, s])
        B.sla_adamw_step(opt, grads, step=t, lr=lr * (1 - (t - 1) / iters), weight_decay=0.0,
                         seed=seed)
        losses.append(loss.detach())
    torch.cuda.synchronize()
    each = (time.perf_counter() - t0) / max(iters - 1, 1) if t0 else None
    losses = torch.stack(losses).cpu().numpy()

    def off(a, b, start):
        return float((a - b).norm() / (b - start).norm())

    out = {"grid": "64x64", "n": n, "steps": steps, "snapshots": snapshots, "bits": bits,
           "iterations": iters, "loss_first": float(losses[0]), "loss_last": float(losses[-1]),
           "rate_error": off(g.detach(), true_g, 3.0),
           "strength_error": off(s.detach(), true_s, 1.0),
           "ms_per_iteration": None if each is None else round(each * 1e3, 3)}
    for h in (A, G):
        h.destroy()
    opt.destroy()
    return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("study", choices=["jacobi", "quality", "trace", "learn"])
    ap.add_argument("--configs", default="0,1,2,3")
    ap.add_argument("--rows", type=int, default=20000)
    ap.add_argument("--iters", type=int, default=300)
    ap.add_argument("--bits", type=int, default=32, choices=[8, 32])
    args = ap.parse_args()
    configs = [int(c) for c in args.configs.split(",")]
    if args.study == "jacobi":
        jacobi(configs)
    elif args.study == "quality":
        quality(configs)
    elif args.study == "learn":
        print(json.dumps(learn(args.iters, args.bits)), flush=True)
    else:
        trace_run(args.rows)


if __name__ == "__main__":
    main()

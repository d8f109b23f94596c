"""Distillation in 64 bits where ids come more than once: an id's probabilities are added up before anything
else is done with them, so that the loss is the divergence of two distributions.

distill64 counts each entry for itself; here it is given one entry an id, x = log Σ e^(t·inv_tau).  What the
kernel's own sum is off by comes on top, u = U32 = 2^-24 each, relative to P = Σ p_k of an id that n entries have:
  - an entry's e^x: x = (t - max)·inv_tau and what is taken from it, 3u·(|x| + |max| + |base|) as in
    distill64, and the exponential 4u, weighted by p_k / P;
  - the sum of n: (n - 1)·u;
  - as a logarithm again: 2u·|log| of the sum (n·e^|x - base| at most), u·|x| of what is stored, and e^x of
    that as any other's.
"""
import torch

from distill_util import distill64
from train_util import U32

F64 = torch.float64


def merged(ids, t, t_lse, inv_tau, V):
    """(ids, t in 64 bits, the relative error of each id's probability) with every id once; absent: -1."""
    B, K = ids.shape
    it = float(torch.tensor(inv_tau, dtype=torch.float32))
    out_ids, out_t, rel = torch.full((B, K), -1), torch.zeros(B, K, dtype=F64), torch.zeros(B, K, dtype=F64)
    for b in range(B):
        here = (ids[b] >= 0) & (ids[b] < V) & (t[b] != -torch.inf)
        if not bool(here.any()):
            continue
        x = t[b][here].double() * it
        one, which = torch.unique(ids[b][here], return_inverse=True)
        base = torch.logsumexp(x, 0) if t_lse is None else t_lse[b].double()
        top = x.max()
        n = torch.zeros(one.numel(), dtype=F64).index_add_(0, which, torch.ones_like(x))
        most = torch.full((one.numel(),), -torch.inf, dtype=F64).scatter_reduce_(0, which, x, "amax")
        e = torch.exp(x - most[which])
        s = torch.zeros(one.numel(), dtype=F64).index_add_(0, which, e)
        off = 3 * U32 * (x.abs() + top.abs() + base.abs()) + 4 * U32
        each = torch.zeros(one.numel(), dtype=F64).index_add_(0, which, e * off) / s
        m = torch.log(s) + most
        r = each + n * U32 + 2 * U32 * ((m - base).abs() + (m - top).abs() + 1) + U32 * m.abs() + 4 * U32
        k = one.numel()
        out_ids[b, :k], out_t[b, :k] = one, m / it
        rel[b, :k] = torch.where(n > 1, r, torch.zeros_like(r))
    return out_ids, out_t, rel


def distill_merged64(z, ids, t, t_lse, inv_tau, dloss=None):
    """(loss, its tolerance, dz, its tolerance without the last rounding) of z [B, V] on the CPU."""
    B, V = z.shape
    it = float(torch.tensor(inv_tau, dtype=torch.float32))
    ids, t, rel = merged(ids, t, t_lse, inv_tau, V)
    loss, loss_tol, dz, dz_tol = distill64(z, ids, t, t_lse, inv_tau, dloss)
    for b in range(B):
        more = rel[b] > 0
        if not bool(more.any()):
            continue
        here = ids[b] >= 0
        at, x, e = ids[b][here], t[b][here] * it, rel[b][here]
        lp = x - (torch.logsumexp(x, 0) if t_lse is None else t_lse[b].double())
        p = torch.exp(lp)
        s = z[b].double() * it
        lse = torch.logsumexp(s, 0)
        e_mass = (p * e).sum()
        w = 1.0 if dloss is None else float(dloss[b].double() * it)
        kept = torch.zeros(V, dtype=torch.bool)
        kept[at] = True
        grad = torch.exp(s - lse) * e_mass
        grad = grad.index_add(0, at, p * e)
        loss_tol[b] += (p * e * ((lp - (s[at] - lse)).abs() + 1)).sum()
        left = s[~kept]
        if t_lse is not None and left.numel():
            p_rest = (1 - p.sum()).clamp_min(1e-12)
            log_q_rest = torch.logsumexp(left, 0) - lse
            loss_tol[b] += 2 * e_mass * ((torch.log(p_rest) - log_q_rest).abs() + 1)
            grad = grad + torch.where(kept, torch.zeros_like(s), torch.exp(s - torch.logsumexp(left, 0)) * e_mass)
        dz_tol[b] += abs(w) * grad
    return loss, loss_tol, dz, dz_tol

"""Distillation in 64 bits, written from its definition, with what the kernels may be off by.

Roundings of the kernels, u = U32 = 2^-24 each (relative to the value):
  - exp((z - m)·c), c = inv_tau·log2 e: the difference, c twice, the product, each off by u of the
    exponent, so e^(4u·|x|) at |x| = |z - m|·inv_tau; the exponential itself 2^-22 = 4u.
  - a sum over V values: a thread adds at most 64 of them in two chains, then 5 levels of a tree over
    lanes, at most 8 in turn and 5 levels over warps and blocks, and 2 peaks: 20 more, and 16 where a block
    takes segments one after another.  Sums are shifted to another largest value by an exponential (where
    that stays the same it is 1): from a thread's to a warp's, a row's, and where a segment has a larger one.
    Teacher: 32 lanes add K / 32 each, 5 levels.
"""
import torch

from train_util import U32

F64 = torch.float64


def distill64(z, ids, t, t_lse, inv_tau, dloss=None):
    """(loss, its tolerance, dz, its tolerance without the last rounding) of z [B, V] on the CPU."""
    B, V = z.shape
    K = ids.shape[1]
    it = float(torch.tensor(inv_tau, dtype=torch.float32))
    z, t = z.double(), t.double()
    loss, loss_tol = torch.zeros(B, dtype=F64), torch.zeros(B, dtype=F64)
    dz, dz_tol = torch.zeros(B, V, dtype=F64), torch.zeros(B, V, dtype=F64)
    w = torch.ones(B, dtype=F64) if dloss is None else dloss.double() * it
    for b in range(B):
        here = (ids[b] >= 0) & (ids[b] < V) & (t[b] != -torch.inf)
        if not bool(here.any()):
            continue
        at, x = ids[b][here], t[b][here] * it
        if t_lse is None:
            base = torch.logsumexp(x, 0)
            e_lp = (K / 32 + 20) * U32 + 3 * U32 * (x.abs() + x.max().abs() + base.abs())
        else:
            base = t_lse[b].double()
            e_lp = 2 * U32 * (x.abs() + base.abs())
        lp = x - base
        p = torch.exp(lp)
        e_p = p * (torch.expm1(e_lp) + 4 * U32)
        s = (z[b] - z[b].max()) * it  # all that follows is the same for s shifted
        lse = torch.log(torch.exp(s).sum())
        kept = torch.zeros(V, dtype=torch.bool)
        kept[at] = True
        far = s[s > -150].abs().max()  # below that e^s is 0 in fp32
        rel = U32 * (32 + 40 + 3 * 4 * float(far) + 6 * 4)  # of a sum, or of q
        mass, e_mass = p.sum(), e_p.sum() + (K / 32 + 10) * U32 * p.sum()
        if t_lse is None:
            e_mass = e_mass + (mass - 1).abs()
        left = s[~kept]
        left = left[left != -torch.inf]
        p_rest, e_rest = torch.zeros((), dtype=F64), torch.zeros((), dtype=F64)
        log_q_rest = torch.full((), -torch.inf, dtype=F64)
        if left.numel():
            log_q_rest = torch.logsumexp(left, 0) - lse
            if t_lse is not None:
                p_rest = (1 - mass).clamp_min(0)
                e_rest = e_mass + U32
        log_q = s[at] - lse
        terms = torch.where(p > 0, p * (lp - log_q), torch.zeros_like(p))
        e_log_q = 3 * U32 * s[at].abs() + rel + 3 * U32 * lse.abs() + U32 * log_q.abs()
        tol = (e_p * (lp - log_q).abs() + p * (e_lp + e_log_q + 2 * U32 * (lp.abs() + log_q.abs()))).sum()
        value = terms.sum()
        tol = tol + (K / 32 + 14) * U32 * terms.abs().sum()
        if p_rest > 0 or e_rest > 0:
            if left.numel():
                near = torch.log((p_rest + e_rest).clamp_min(1e-12)) - log_q_rest
                if p_rest > 0:
                    value = value + p_rest * (torch.log(p_rest) - log_q_rest)
                    near = torch.maximum(near.abs(), (torch.log(p_rest) - log_q_rest).abs())
                tol = tol + e_rest * (near.abs() + 2) + (p_rest + e_rest) * (2 * rel + 6 * U32 * (log_q_rest.abs() + 1))
        loss[b], loss_tol[b] = value, tol + U32 * value.abs()
        q = torch.exp(s - lse)
        M, e_M = mass + p_rest, e_mass + e_rest
        P = torch.zeros(V, dtype=F64).index_add_(0, at, p)
        e_P = torch.zeros(V, dtype=F64).index_add_(0, at, e_p + K * U32 * p)
        share = torch.zeros(V, dtype=F64)  # q / q_rest
        if left.numel():
            share = torch.exp(s - left.max())
            share = share / share[~kept].sum()
        d = torch.where(kept, M * q - P, M * q - p_rest * share)
        e_kept = M * q * (2 * rel + 4 * U32) + q * e_M + e_P + 2 * U32 * (M * q + P)
        e_left = M * q * (3 * rel + 6 * U32) + q * e_M + share * e_rest + (3 * rel + 4 * U32) * (M * q + p_rest * share)
        dz[b] = w[b] * d
        dz_tol[b] = w[b].abs() * torch.where(kept, e_kept, e_left) + 3 * U32 * dz[b].abs() + 1e-37
    return loss, loss_tol, dz, dz_tol

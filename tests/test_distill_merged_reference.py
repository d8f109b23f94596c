"""The 64-bit form of distillation with repeated ids (distill_merged_util) against its definition: probabilities
by id over the whole vocabulary, autograd, and what a divergence has to be."""
import torch

from distill_merged_util import distill_merged64
from distill_util import distill64

F64 = torch.float64


def dense(z, ids, t, t_lse, it):
    """The loss from P over the vocabulary."""
    x = t.double() * it
    base = torch.logsumexp(x, 1) if t_lse is None else t_lse.double()
    P = torch.zeros_like(z).scatter_add(1, ids, torch.exp(x - base[:, None]))
    logq = torch.log_softmax(z * it, 1)
    kept = torch.zeros_like(z).scatter(1, ids, 1.0) > 0
    loss = torch.where(kept, P * (torch.log(P.clamp_min(1e-300)) - logq), torch.zeros_like(z)).sum(1)
    if t_lse is not None:
        rest = 1 - P.sum(1)
        q_rest = torch.where(kept, torch.zeros_like(z), torch.exp(logq)).sum(1)
        loss = loss + rest * (torch.log(rest) - torch.log(q_rest))
    return loss


def test_repeated_ids_against_the_dense_form():
    for rest in (False, True):
        g = torch.Generator().manual_seed(3)
        B, V, K = 5, 40, 12
        z = torch.randn(B, V, generator=g, dtype=F64) * 2
        ids = torch.randint(0, 9, (B, K), generator=g)
        ids[4] = 7
        t = torch.randn(B, K, generator=g)
        t_lse = (torch.logsumexp(t.double() * 0.5, 1) + 0.3).float() if rest else None
        w = torch.tensor([1.0, 0.5, 2.0, -1.0, 1.0])
        loss, _, dz, _ = distill_merged64(z, ids, t, t_lse, 0.5, w)
        zz = z.clone().requires_grad_(True)
        want = dense(zz, ids, t, t_lse, 0.5)
        (gz,) = torch.autograd.grad((want * w.double()).sum(), zz)
        assert torch.allclose(loss, want.detach(), rtol=1e-11, atol=1e-12)
        assert torch.allclose(dz, gz, rtol=1e-10, atol=1e-13)
        assert bool((loss >= 0).all())


def test_an_id_cut_in_two_is_the_id():
    """Two entries of half the probability are one of all of it; entries for themselves are off by the entropy
    of the split, log 2 here, and negative."""
    z = torch.tensor([[0.0, 0.0, 3.0, 0.0]], dtype=F64)
    one = distill64(z, torch.tensor([[2]]), torch.zeros(1, 1), None, 1.0)
    two = distill_merged64(z, torch.tensor([[2, 2]]), torch.zeros(1, 2), None, 1.0)
    assert torch.allclose(one[0], two[0]) and torch.allclose(one[2], two[2])
    assert abs(float(two[0]) + float(torch.log_softmax(z, 1)[0, 2])) < 1e-12
    apart = distill64(z, torch.tensor([[2, 2]]), torch.zeros(1, 2), None, 1.0)
    assert float(apart[0]) < 0 and abs(float(two[0] - apart[0]) - float(torch.log(torch.tensor(2.0)))) < 1e-6


def test_distinct_ids_are_left_as_they_are():
    g = torch.Generator().manual_seed(4)
    z, t = torch.randn(3, 30, generator=g, dtype=F64), torch.randn(3, 5, generator=g)
    ids = torch.stack([torch.randperm(30, generator=g)[:5] for _ in range(3)])
    ids[1, 2], ids[2] = -1, 30
    a, b = distill64(z, ids, t, None, 1.0), distill_merged64(z, ids, t, None, 1.0)
    assert torch.allclose(a[0], b[0]) and torch.allclose(a[2], b[2])
    assert torch.allclose(a[1], b[1], rtol=1e-3) and torch.allclose(a[3], b[3], rtol=1e-3)

"""The 64-bit form of distillation (distill_util) against its definition taken apart: autograd, cross
entropy, differences."""
import torch

from distill_util import distill64

F64 = torch.float64


def case(seed, B, V, K, rest):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(B, V, generator=g, dtype=F64) * 2
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(B)])
    t = torch.randn(B, K, generator=g, dtype=F64).float()
    t_lse = (torch.logsumexp(t.double() * 0.5, 1) + 0.3).float() if rest else None
    return z, ids, t, t_lse


def loss_of(z, ids, t, t_lse, it):
    logq = torch.log_softmax(z * it, 1)
    base = torch.logsumexp(t.double() * it, 1) if t_lse is None else t_lse.double()
    p = torch.exp(t.double() * it - base[:, None])
    loss = (p * (torch.log(p) - logq.gather(1, ids))).sum(1)
    if t_lse is not None:
        rest = 1 - p.sum(1)
        q_rest = torch.exp(logq).scatter(1, ids, 0.0).sum(1)
        loss = loss + rest * (torch.log(rest) - torch.log(q_rest))
    return loss


def test_loss_and_gradient_by_autograd_and_differences():
    for rest in (False, True):
        z, ids, t, t_lse = case(3, 4, 50, 7, rest)
        w = torch.tensor([1.0, 0.5, 2.0, -1.0])
        loss, _, dz, _ = distill64(z, ids, t, t_lse, 0.5, w)
        zz = z.clone().requires_grad_(True)
        want = loss_of(zz, ids, t, t_lse, 0.5)
        assert torch.allclose(loss, want.detach(), rtol=1e-12, atol=1e-13)
        (g,) = torch.autograd.grad((want * w.double()).sum(), zz)
        assert torch.allclose(dz, g, rtol=1e-11, atol=1e-14)
        v = torch.randn(4, 50, generator=torch.Generator().manual_seed(1), dtype=F64)
        h = 1e-5
        diff = (distill64(z + h * v, ids, t, t_lse, 0.5, w)[0] - distill64(z - h * v, ids, t, t_lse, 0.5, w)[0]) / (2 * h)
        assert torch.allclose((dz * v).sum(1), diff * w.double(), rtol=1e-7, atol=1e-9)


def test_one_entry_is_cross_entropy():
    z, ids, t, _ = case(4, 5, 33, 1, False)
    loss, _, dz, _ = distill64(z, ids, t, None, 1.0, torch.ones(5))
    assert torch.allclose(loss, torch.nn.functional.cross_entropy(z, ids[:, 0], reduction="none"))
    q = torch.softmax(z, 1).scatter_add(1, ids, -torch.ones(5, 1, dtype=F64))
    assert torch.allclose(dz, q)


def test_absent_and_repeated_entries():
    z, ids, t, _ = case(5, 3, 20, 4, False)
    ids[0] = -1
    ids[1, 2:] = torch.tensor([20, -7])
    loss, _, dz, _ = distill64(z, ids, t, None, 1.0)
    assert float(loss[0]) == 0 and not bool(dz[0].any())
    two = distill64(z[1:2], ids[1:2, :2], t[1:2, :2], None, 1.0)
    assert torch.allclose(loss[1:2], two[0]) and torch.allclose(dz[1:2], two[2])
    # the same id twice: its probabilities add up in the gradient
    again = distill64(z[2:], ids[2:, [0, 1, 0]], t[2:, [0, 1, 0]], None, 1.0)
    p = torch.softmax(t[2, [0, 1, 0]].double(), 0)
    q = torch.softmax(z[2], 0)
    q[ids[2, 0]] -= p[0] + p[2]
    q[ids[2, 1]] -= p[1]
    assert torch.allclose(again[2][0], q)

"""Distillation where ids come more than once, on the GPU: an id has the sum of its entries' probabilities, in the
loss as in the gradient (distill_merged_util)."""
import math

import pytest
import torch

from distill_merged_util import distill_merged64
from gpu_util import cuda_ok
from test_distill_gpu import call, make, up8
from train_util import HALF_BF16, U32, Guarded, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32 = torch.bfloat16, torch.float32


def check(d, out, dz, inv_tau):
    loss, l_tol, want, tol = distill_merged64(d["z"], d["ids"], d["t"], d["t_lse"], inv_tau, d["dloss"])
    if out is not None:
        within(out, loss, l_tol, "loss")
    if dz is not None:
        half = HALF_BF16 if dz.dtype == BF else U32
        within(dz[:, :want.shape[1]], want, 1.01 * tol + half * want.abs(), "dz")


def repeat(d, how, V, seed):
    B, K = d["ids"].shape
    g = torch.Generator().manual_seed(seed)
    ids = d["ids"]
    if how == "halves":
        ids[:, K // 2:] = ids[:, :K - K // 2].clone()
    elif how == "pairs":
        ids[:, 1::2] = ids[:, 0:2 * (K // 2):2].clone()
    elif how == "one":
        ids[:] = ids[:, :1].clone()
    elif how == "few":  # drawn from a few, some of them absent
        few = torch.stack([torch.randperm(V, generator=g)[:max(1, K // 3)] if V >= K // 3 else
                           torch.arange(max(1, K // 3)) % V for _ in range(B)])
        ids[:] = few.gather(1, torch.randint(0, few.shape[1], (B, K), generator=g))
        ids[::2, ::5] = -1
        d["t"][1::2, 3::7] = -math.inf
    else:  # "last": the first of all comes again at the end
        ids[:, -1] = ids[:, 0]
    if d["t_lse"] is not None:
        t = torch.where((ids >= 0) & (d["t"] != -math.inf), d["t"], torch.full_like(d["t"], -1e30))
        d["t_lse"] = torch.logsumexp(t, 1) + 0.05 + 0.3 * torch.rand(B, generator=g)
    return d


SHAPES = [(1, 1, 2), (3, 5, 9), (4, 50, 33), (2, 9, 1024), (5, 1000, 64), (2, 32000, 1024), (2, 70001, 300),
          (3, 131072, 130), (2, 262144, 1001), (304, 40009, 5), (330, 300, 17)]


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("how", ["halves", "pairs", "one", "few", "last"])
@pytest.mark.parametrize("B,V,K", SHAPES)
def test_loss_and_gradient(B, V, K, how, dt, rest):
    d = repeat(make(V + K, B, V, K, dt, rest), how, V, K)
    g = Guarded()
    out, dz, _ = call(d, up8(V), 1.0, g)
    alone, _, _ = call(d, up8(V), 1.0, g, grad=False)
    torch.cuda.synchronize()
    g.check()
    check(d, out, dz, 1.0)
    check(d, alone, None, 1.0)
    _, here, _ = call(d, up8(V), 1.0, g, in_place=True, loss=False)
    again, _, _ = call(d, up8(V), 1.0, g, grad=False)
    g.check()
    assert torch.equal(here[:, :V], dz[:, :V]) and torch.equal(again, alone)


@pytest.mark.parametrize("V", [4, 70000])
@pytest.mark.parametrize("n", [2, 3, 600])
def test_an_id_cut_into_equal_parts_is_the_id(V, n):
    """n entries of one id with the same t: cross entropy with it."""
    z = torch.zeros(1, V)
    z[0, 2] = 3.0
    d = dict(z=z, ids=torch.full((1, n), 2), t=torch.full((1, n), -1.5), t_lse=None, dloss=torch.ones(1))
    g = Guarded()
    out, dz, _ = call(d, up8(V), 1.0, g)
    q = torch.softmax(z.double(), 1)
    _, l_tol, _, tol = distill_merged64(d["z"], d["ids"], d["t"], None, 1.0, d["dloss"])
    within(out, -torch.log(q[:, 2]), l_tol, "loss")
    q[0, 2] -= 1
    within(dz[:, :V], q, 1.01 * tol + U32 * q.abs(), "dz")


@pytest.mark.parametrize("rest", [False, True])
def test_probabilities_that_underflow(rest):
    """Entries far below the others, and ids that have only such: they count as nothing."""
    B, V, K = 3, 900, 40
    d = make(21, B, V, K, F32, rest)
    d["ids"][:, 20:] = d["ids"][:, :20].clone()
    d["t"][1, 20:] = -4e4  # beside one that counts
    d["t"][2, 7] = d["t"][2, 27] = -3e38  # alone
    if rest:
        d["t_lse"] = torch.logsumexp(d["t"], 1) + 0.2
    g = Guarded()
    out, dz, _ = call(d, up8(V), 1.0, g)
    g.check()
    far = {**d, "t": d["t"].clamp_min(-1e3)}
    check(far, out, dz, 1.0)
    alone, _, _ = call(d, up8(V), 1.0, g, grad=False)
    check(far, alone, None, 1.0)


@pytest.mark.parametrize("B,V,K", [(700, 32000, 40), (40, 131072, 600), (400, 65536, 64)])
def test_many_rows_some_with_repeats(B, V, K):
    """Rows with and without repeats in turn, through the same blocks: each as it is alone."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(B, V, device="cuda", generator=g).to(BF)
    ids = torch.randint(0, V, (B, K), device="cuda", generator=g)
    ids[::3, 5:] = ids[::3, :-5].clone()
    ids[1::7] = -1
    t = torch.randn(B, K, device="cuda", generator=g)
    lse, dl = torch.logsumexp(t, 1) + 0.1, torch.rand(B, device="cuda", generator=g)
    loss, fwd, dz = torch.empty(B, device="cuda"), torch.empty(B, device="cuda"), torch.empty_like(z)
    mhc.mhc_distill_loss_backward(z, V, ids, t, lse, 1.0, dl, B, V, K, loss, dz)
    mhc.mhc_distill_loss(z, V, ids, t, lse, 1.0, B, V, K, fwd)
    rows = list(range(12)) + list(range(B - 12, B))
    d = dict(z=z[rows].cpu(), ids=ids[rows].cpu(), t=t[rows].cpu(), t_lse=lse[rows].cpu(), dloss=dl[rows].cpu())
    check(d, loss[rows], dz[rows], 1.0)
    check(d, fwd[rows], None, 1.0)
    one, dz1 = torch.empty(1, device="cuda"), torch.empty(1, V, dtype=BF, device="cuda")
    for b in range(0, B, B // 10):
        part = [v[b:b + 1].clone() for v in (z, ids, t, lse, dl)]
        mhc.mhc_distill_loss_backward(part[0], V, *part[1:4], 1.0, part[4], 1, V, K, one, dz1)
        d = dict(zip(("z", "ids", "t", "t_lse", "dloss"), (v.cpu() for v in part)))
        check(d, one, dz1, 1.0)
        check(d, loss[b:b + 1], dz[b:b + 1], 1.0)

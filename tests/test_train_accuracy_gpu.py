"""How near the training gradients come to their 64-bit values where one term, or the far end of a
range, would hide in the others' rounding."""
import pytest
import torch

from gpu_util import cuda_ok
from test_train_gpu import ALPHA, pre_case, pre_run
from train_util import HALF_BF16, MMA_STEP, U32, Guarded, sinkhorn64, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")


@pytest.mark.parametrize("B,n,C", [(70, 1, 200), (130, 2, 72), (65, 3, 264), (200, 4, 136), (67, 5, 96),
                                   (66, 6, 264), (131, 7, 72), (129, 8, 136), (70, 8, 288)])
def test_the_projections_share_of_dX(B, n, C):
    """dX = Σ_k dY[k]·φ[k] alone: what is left of dY in this product is 2^-16 of it, so that a result
    small against its terms is as near as a large one."""
    d = pre_case(B + 7 * n, B, n, C, 0)
    for k in ("G", "dF", "Y"):
        d[k] = torch.zeros_like(d[k])
    out, _ = pre_run(d, B, n, C, 0, Guarded())
    N = n * n + 2 * n
    f = {k: v.double() for k, v in d.items() if k not in ("q", "s")}
    # H̃ is the bias where Y is zero, and without a Sinkhorn step dH̃_res = exp(H̃)·dH_res
    Ht = f["bias"][2 * n:].view(n, n)
    dHt = torch.cat([torch.zeros(B, n, dtype=torch.float64), f["dhq"] * f["hq"] * (1 - f["hq"] / 2),
                     (torch.exp(Ht) * f["dhr"]).view(B, n * n)], 1)
    # the sigmoid's products of values that are exact; exp within 2 roundings and its product
    t_H = torch.cat([torch.zeros(B, n, dtype=torch.float64), 6 * U32 * (f["dhq"] * f["hq"]).abs(),
                     4 * U32 * dHt[:, 2 * n:].abs()], 1)
    al = torch.tensor([ALPHA[0]] * n + [ALPHA[1]] * n + [ALPHA[2]] * n * n, dtype=torch.float64)
    dY, t_Y = al * dHt / f["r"][:, None], al * t_H / f["r"][:, None]
    t_Y = t_Y + 4 * U32 * dY.abs()
    ref = (dY @ f["phi"]).view(B, n, C)
    terms = (dY.abs() @ f["phi"].abs()).view(B, n, C)
    steps = 2 * ((N + 15) // 16)  # two bf16 terms of dY
    tol = (HALF_BF16 * ref.abs() + 1.01 * (2.0 ** -16 + MMA_STEP * steps) * terms +
           1.01 * (t_Y @ f["phi"].abs()).view(B, n, C))
    within(out["dX"], ref, tol, "dX")


@pytest.mark.parametrize("n", [2, 3, 4, 5, 6, 7, 8])
def test_sinkhorn_of_widely_spread_logits(n):
    """H̃_res of standard deviation 40: wherever the forward is finite the backward is, and a token whose
    block fp32 can hold has the gradient of the iteration."""
    B, C, iters, dev = 20000, 8, 20, "cuda"
    K, N = n * C, n * n + 2 * n
    gen = torch.Generator(device=dev).manual_seed(n)
    rnd = lambda *s, std=1.0: torch.randn(*s, device=dev, generator=gen) * std  # noqa: E731
    Ht = rnd(B, n, n, std=40.0)
    Y = torch.cat([rnd(B, 2 * n), Ht.view(B, n * n) / ALPHA[2]], 1)
    r, bias = torch.ones(B, device=dev), torch.zeros(N, device=dev)
    H = [torch.empty(B, n, device=dev), torch.empty(B, n, device=dev), torch.empty(B, n, n, device=dev)]
    mhc.mhc_coeffs(Y, r, *ALPHA, bias, iters, B, n, *H)
    dead = ~torch.isfinite(H[2]).flatten(1).all(1)
    assert float(dead.float().mean()) < 0.02  # a column that fp32's exp does not reach
    Y[dead] = 0
    mhc.mhc_coeffs(Y, r, *ALPHA, bias, iters, B, n, *H)
    assert bool(torch.isfinite(H[2]).all())
    phi, D = rnd(N, K, std=0.05).to(torch.bfloat16), rnd(B, n, n, std=0.1)
    zeros = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=dev)  # noqa: E731
    q, s = zeros(B, n, C, dtype=torch.uint8), torch.full((B, n, 1), 10, dtype=torch.uint8, device=dev)
    dX, dphi = zeros(B, n, C), zeros(N, K, dtype=torch.float32)
    dbias, dalpha = zeros(N, dtype=torch.float32), zeros(3, dtype=torch.float32)
    mhc.mhc_pre_backward(zeros(B, n, C), zeros(B, C), q, s, phi, *ALPHA, bias, iters, Y, r, *H, D,
                         zeros(B, n, dtype=torch.float32), 0, B, n, C, dX, dphi, dbias, dalpha,
                         mhc.pre_backward_workspace(B, n, C, iters))
    for k, t in (("dX", dX), ("dphi", dphi), ("dbias", dbias), ("dalpha", dalpha)):
        assert bool(torch.isfinite(t).all()), "%s: %d not finite" % (k, int((~torch.isfinite(t)).sum()))
    h = (ALPHA[2] * Y[:, 2 * n:].double()).view(B, n, n).requires_grad_(True)
    with torch.enable_grad():
        dHt = torch.autograd.grad(sinkhorn64(h, iters), h, D.double())[0].view(B, n * n)
    h = h.detach()
    # every column's largest entry after the row shift is far above fp32's smallest number
    fair = (h - h.amax(-1, keepdim=True)).amax(-2).amin(-1) > -60
    assert float(fair.float().mean()) > 0.5
    # 4·iters + 4 half steps of n + 8 roundings, of entries at most 1, whose logits are off by roundings too
    t_H = (4 * iters + 4) * (n + 8) * U32 * D.double().abs().sum((1, 2)) * (1 + h.abs().amax((1, 2)))
    f = phi.double()[2 * n:]
    ref, terms = ALPHA[2] * dHt @ f, ALPHA[2] * dHt.abs() @ f.abs()
    tol = (HALF_BF16 * ref.abs() + 1.01 * (2.0 ** -16 + MMA_STEP * 2 * ((N + 15) // 16) + 4 * U32) * terms +
           1.01 * ALPHA[2] * t_H[:, None] * f.abs().sum(0))
    within(dX.view(B, K)[fair], ref[fair].cpu(), tol[fair].cpu(), "dX")

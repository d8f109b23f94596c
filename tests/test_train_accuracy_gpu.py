"""How near the training gradients come to their 64-bit values where one term, or the far end of a
range, would hide in the others' rounding."""
import pytest
import torch

from gpu_util import cuda_ok
from test_train_gpu import ALPHA, pre_case, pre_run
from train_util import HALF_BF16, MMA_STEP, U32, Guarded, within

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

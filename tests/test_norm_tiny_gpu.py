"""The norm's backward where rstd² is no number of fp32: rows of 1e-20 with eps = 0 (or as small), and rows of
zeros under a tiny eps."""
import pytest
import torch

from gpu_util import cuda_ok
from test_norm_gpu import back64
from test_train_gpu import normal
from train_util import HALF_BF16, Guarded, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32 = torch.bfloat16, torch.float32


def backward(d, skip):
    B, C = d["H"].shape
    g = Guarded()
    dev = {k: g.put(v) for k, v in d.items()}
    dH, dgain = g.empty(B, C, dtype=BF), g.empty(C)
    mhc.mhc_rmsnorm_backward(dev["dZ"], dev["H"], dev["gain"], dev["rstd"], dev["skip"] if skip else None, 0, B, C, dH,
                             dgain, mhc.rmsnorm_backward_workspace(B, C))
    torch.cuda.synchronize()
    g.check()
    return dH, dgain


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("B,C", [(5, 72), (33, 1000), (3, 8200)])
def test_tiny_rows(B, C, skip):
    """Every other row tiny, its rstd that of eps = 0 in 64 bits, rounded."""
    H = normal(1, B, C)
    H[::2] *= 2.0 ** -66  # 1.4e-20; the others are ordinary rows
    d = dict(H=H, dZ=normal(2, B, C, std=1e-2), skip=normal(3, B, C, std=1e-2), gain=1 + normal(4, C, std=0.2, dtype=F32))
    d["rstd"] = torch.where(torch.arange(B) % 2 == 0, 2.0 ** 66, 1.0) * d["H"].double().mul(
        torch.where(torch.arange(B) % 2 == 0, 2.0 ** 66, 1.0)[:, None]).square().mean(1).rsqrt()
    d["rstd"] = d["rstd"].float()
    assert bool((d["rstd"][::2] > 1.85e19).all()) and not bool(torch.isfinite(d["rstd"][::2].square()).any())
    dH, dgain = backward(d, skip)
    want, tol, wg, wg_tol = back64(d, skip)
    # t·H is about 1e-22: its products and their sum are normal numbers of fp32
    within(dH, want, HALF_BF16 * want.abs() + 1.01 * tol, "dH")
    within(dgain, wg, wg_tol, "dgain")


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 2e-39, 1e-38])
def test_forward_and_backward_of_zeros_and_tiny_rows(eps):
    """Zeros stay zeros; every gradient that fp32 and bf16 hold is a number."""
    B, C = 6, 264
    A = normal(5, B, C)
    A[1] = 0
    A[2] *= 2.0 ** -66
    A[4] = 0
    dZ = normal(6, B, C, std=1e-2)
    dZ[1] = 0
    gain = torch.ones(C, device="cuda")
    Z, H, rstd = torch.empty(B, C, dtype=BF, device="cuda"), A.cuda(), torch.empty(B, device="cuda")
    R = torch.zeros(B, C, dtype=BF, device="cuda")
    mhc.mhc_add_rmsnorm(A.cuda(), R, gain, eps, B, C, H, rstd, Z)
    assert bool(torch.isfinite(rstd).all()) and bool(torch.isfinite(Z.float()).all()) and not bool(Z[[1, 4]].any())
    dH, dgain = backward(dict(H=H.cpu(), rstd=rstd.cpu(), dZ=dZ, gain=gain.cpu(), skip=dZ), False)
    assert bool(torch.isfinite(dH.float()).all()) and bool(torch.isfinite(dgain).all())
    assert not bool(dH[1].any())  # padding: no gradient in, none out
    want, tol, _, _ = back64(dict(H=H.cpu(), rstd=rstd.cpu(), dZ=dZ, gain=gain.cpu()), False)
    within(dH, want, HALF_BF16 * want.abs() + 1.01 * tol, "dH")

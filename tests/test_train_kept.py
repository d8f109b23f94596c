"""How far the 8-bit form of X is from X, as include/mhc.h states it."""
import pytest
import torch

from gpu_util import cuda_ok
from train_util import pack64, unpack64

BF = torch.bfloat16


def blocks():
    """Blocks of 32 by their largest magnitude: around the ends of (224, 448] times a power of two, at the
    ends of the scale's range, and where the scale is at its smallest; values from there down by 2^-20."""
    g = torch.Generator().manual_seed(1)
    tops = [225.0, 224.0, 226.0, 300.0, 448.0, 450.0, 1.0, 1.75, 1.7578125]
    tops = [t * 2.0 ** e for t in tops for e in (-100, -9, 0, 40)]
    tops += [448 * 2.0 ** -117, 225 * 2.0 ** -117, 3 * 2.0 ** -117, 2.0 ** -126, 1.5 * 2.0 ** 126]
    rows = []
    for t in tops:
        for lo in (0.0, -8.0, -13.0, -20.0):
            x = t * torch.exp2(lo * torch.rand(32, generator=g, dtype=torch.float64))
            x = x * (1 - 2 * torch.randint(0, 2, (32,), generator=g))
            x[0] = t
            rows.append(x)
    return torch.stack(rows).to(BF).view(len(rows), 1, 32)


def check(X, q, s):
    x, kept = X.double(), unpack64(q, s)
    scale = torch.exp2(s.double().cpu() - 127)
    off = (kept - x).abs()
    normal = x.abs() >= 2.0 ** -6 * scale
    assert bool((off <= torch.where(normal, 2.0 ** -4 * x.abs(), 2.0 ** -10 * scale)).all())
    near = x.abs() >= 2.0 ** -13 * x.abs().amax(-1, keepdim=True)
    assert bool(normal[near & (s > 10)].all())
    return off, x


def test_the_bound_of_the_definition():
    X = blocks()
    off, x = check(X, *pack64(X))
    # and no wider: within 2^-15 of the largest the relative bound does not hold
    amax = x.abs().amax(-1, keepdim=True)
    assert bool(((off > 2.0 ** -4 * x.abs()) & (x.abs() >= 2.0 ** -15 * amax) & (amax > 2.0 ** -100)).any())


@pytest.mark.gpu
@pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")
def test_the_bound_of_the_kernel():
    import gemm_rms_sinkhorn_gb300 as mhc

    X = blocks()
    B = X.shape[0]
    q, s = mhc.alloc_kept(B, 1, 32)
    mhc.mhc_ckpt_pack(X.cuda(), B, 1, 32, q, s)
    check(X, q.cpu(), s.cpu())
    back = torch.empty(B, 1, 32, dtype=BF, device="cuda")
    mhc.mhc_ckpt_unpack(q, s, B, 1, 32, back)
    assert torch.equal(back.double().cpu(), unpack64(q, s))

"""Distillation of rows that have no loss: their loss is NaN, with and without the teacher's sum, and the rows
beside them are what they are alone."""
import math

import pytest
import torch

from distill_util import distill64
from gpu_util import cuda_ok
from test_distill_gpu import call, make, up8
from train_util import HALF_BF16, U32, Guarded, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


def run(d, V, inv_tau=1.0):
    """The losses of both calls, which agree on what is NaN, and dz [B, V]."""
    g = Guarded()
    out, dz, _ = call(d, up8(V), inv_tau, g)
    alone, _, _ = call(d, up8(V), inv_tau, g, grad=False)
    torch.cuda.synchronize()
    g.check()
    assert torch.equal(torch.isnan(out), torch.isnan(alone))
    return out, alone, dz[:, :V]


def others(d, out, alone, dz, rows, inv_tau=1.0):
    part = {k: (v[rows] if v is not None else None) for k, v in d.items()}
    loss, l_tol, want, tol = distill64(part["z"], part["ids"], part["t"], part["t_lse"], inv_tau, part["dloss"])
    within(out[rows], loss, l_tol, "loss")
    within(alone[rows], loss, l_tol, "loss alone")
    within(dz[rows], want, 1.01 * tol + (HALF_BF16 if dz.dtype == BF else U32) * want.abs(), "dz")


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V,K", [(900, 5), (70000, 40), (262144, 3)])
def test_a_teacher_that_is_not_finite(V, K, dt, rest):
    d = make(3, 6, V, K, dt, rest)
    d["t"][1, K - 1] = INF
    d["t"][2, 0] = NAN
    d["t"][3] = INF
    d["t"][4, 1] = NAN
    d["ids"][4, 0] = -1
    out, alone, dz = run(d, V)
    assert torch.isnan(out).tolist() == [False, True, True, True, True, False]
    others(d, out, alone, dz, [0, 5])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [900, 70000])
def test_probabilities_past_fp32(V, dt):
    """Finite logits whose e^(t·inv_tau - t_lse) is no number of fp32: by the product, by the difference."""
    d = make(4, 4, V, 6, dt, True, 4.0)
    d["t"][1, 2] = 1e38  # times 4 it is +inf
    d["t"][2, 3] = float(d["t_lse"][2]) / 4 + 30.0  # e^120
    out, alone, dz = run(d, V, 4.0)
    assert torch.isnan(out).tolist() == [False, True, True, False]
    others(d, out, alone, dz, [0, 3], 4.0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V,K", [(900, 5), (70000, 40), (24, 24)])
def test_logits_without_a_distribution_under_a_teacher_that_keeps_nothing(V, K, dt):
    """Every p underflows, so that no term of the loss sees z: all -inf, and a NaN or +inf with nothing left
    over beside it."""
    d = make(5, 6, V, K, dt, True)
    d["t_lse"][1:5] = 1e4
    d["z"][1] = -INF
    d["z"][2] = -INF
    d["z"][2, d["ids"][2, 0]] = NAN
    d["z"][3] = -INF
    d["z"][3, d["ids"][3, 1]] = INF
    d["ids"][4] = -1  # no entries: nothing at all
    d["z"][4] = -INF
    out, alone, dz = run(d, V)
    assert torch.isnan(out).tolist() == [False, True, True, True, False, False]
    assert bool(torch.isnan(dz[1:4]).all())
    assert float(out[4]) == 0.0 and not bool(dz[4].any())
    others(d, out, alone, dz, [0, 5])

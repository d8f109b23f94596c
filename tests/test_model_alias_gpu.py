"""The norms where inputs are one buffer, in place too, and the model's end on two streams at once into buffers
that hold nothing of the answer."""
import pytest
import torch

from gpu_util import cuda_ok
from test_model_run_gpu import End
from test_norm_gpu import EPS, back64, back_case, check_outputs, outputs
from test_train_gpu import normal, streams
from train_util import HALF_BF16, U32, Guarded, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,C", [(1, 8), (77, 1000), (700, 2056), (3, 16384)])
def test_a_sum_of_one_buffer_with_itself(B, C, q8, in_place):
    A, gain = streams(B + C, B, 1, C)[:, 0], 1 + normal(1, C, std=0.2, dtype=F32)
    g = Guarded()
    Ad = g.put(A)
    H, rstd, Z = outputs(g, B, C, q8, True)
    H = Ad if in_place else H
    (mhc.mhc_add_rmsnorm_q8 if q8 else mhc.mhc_add_rmsnorm)(Ad, Ad, g.put(gain), EPS, B, C, H, rstd, *Z)
    torch.cuda.synchronize()
    g.check()
    H64 = 2 * A.double()
    check_outputs(H, rstd, Z, H64, gain, EPS, U32 * H64.abs())


@pytest.mark.parametrize("all_one", [False, True])
@pytest.mark.parametrize("B,C", [(5, 72), (300, 1000), (3, 16384)])
def test_a_gradient_that_is_both_of_the_backwards(B, C, all_one):
    """dZ, dH_skip and dH one buffer; and H that buffer, too."""
    d = back_case(B + C, B, C)
    if all_one:
        d["dZ"] = d["H"]
    d["skip"] = d["dZ"]
    g = Guarded()
    dev = {k: g.put(v) for k, v in d.items()}
    dgain = g.empty(C)
    ws = mhc.rmsnorm_backward_workspace(B, C)
    mhc.mhc_rmsnorm_backward(dev["dZ"], dev["dZ"] if all_one else dev["H"], dev["gain"], dev["rstd"], dev["dZ"], 0, B, C, dev["dZ"], dgain, ws)
    torch.cuda.synchronize()
    g.check()
    want, tol, wg, wg_tol = back64(d, True)
    within(dev["dZ"], want, HALF_BF16 * want.abs() + 1.01 * tol, "dH")
    within(dgain, wg, wg_tol, "dgain")


def test_two_streams_at_once_over_cleared_outputs():
    """As test_two_streams_at_once of the model's end, but each run has to write all of its outputs; what stands
    in the logits' columns past V is no number."""
    pair = [End(60, 4, 1000, 33001, 20, seed) for seed in (1, 2)]
    outs = lambda m: [t[:, :m.size[3]] if t is m.z else t for t in m.outputs()]  # noqa: E731
    for m in pair:
        m.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs(m)] for m in pair]
    lanes = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(5):
        for m in pair:
            for t in (m.H, m.Z, m.rstd, m.z, m.loss, m.dz, m.dH, m.dgain, m.q, m.s, m.Zq, m.Zsum, m.ws):
                t.view(torch.uint8).fill_(0xFF)
        torch.cuda.synchronize()
        for m, lane in zip(pair, lanes):
            with torch.cuda.stream(lane):
                m.run()
        torch.cuda.synchronize()
        for m, w in zip(pair, want):
            for i, (a, b) in enumerate(zip(outs(m), w)):
                assert torch.equal(a, b), (turn, i)

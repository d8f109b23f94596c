"""The waits of the dX and dφ pipelines give up without a fault: a unit of CTA 0 is left without its copies
(include/mhc_testing.h) and the limit is 50 ms.  The call reports MHC_ERR_TIMEOUT through the status word,
and the next one is what it would have been."""
import pytest
import torch

from gpu_util import cuda_ok
from test_train_gpu import ALPHA

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32 = torch.bfloat16, torch.float32


def case(B, n, C):
    N, K, gen = n * n + 2 * n, n * C, torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s, dtype=F32, std=1.0: torch.randn(*s, device="cuda", generator=gen, dtype=dtype) * std  # noqa: E731
    q, s = mhc.alloc_kept(B, n, C)
    mhc.mhc_ckpt_pack(rnd(B, n, C, dtype=BF), B, n, C, q, s)
    h = torch.rand(B, n * n + 2 * n, device="cuda", generator=gen)
    ins = [rnd(B, n, C, dtype=BF), rnd(B, C, dtype=BF), q, s, rnd(N, K, dtype=BF, std=0.05)]
    rest = [rnd(B, N), rnd(B).abs() + 0.5, h[:, :n].contiguous(), h[:, n:2 * n].contiguous(),
            h[:, 2 * n:].contiguous(), rnd(B, n * n, std=0.1), rnd(B, n, std=0.1)]
    return ins, rnd(N, std=0.3), rest


def run(c, B, n, C, iters, stall=None):
    """The outputs; stall: (kernel, unit, limit)."""
    ins, bias, rest = c
    N, K = n * n + 2 * n, n * C
    out = [torch.zeros(B, n, C, dtype=BF, device="cuda"), torch.zeros(N, K, device="cuda"),
           torch.zeros(N, device="cuda"), torch.zeros(3, device="cuda")]
    ws = mhc.pre_backward_workspace(B, n, C, iters)
    if stall is None:
        mhc.mhc_pre_backward(*ins, *ALPHA, bias, iters, *rest, 0, B, n, C, *out, ws)
    else:
        p = lambda ts: [t.data_ptr() for t in ts]  # noqa: E731
        st = mhc._lib.mhc_testing_pre_backward_stalled(
            *p(ins), *ALPHA, bias.data_ptr(), iters, *p(rest), 0, B, n, C, *p(out), ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream, *stall)
        assert st == mhc.MHC_OK, mhc.mhc_status_str(st)
    torch.cuda.synchronize()  # a fault would raise here
    return out


# several units a CTA; codes copied by TMA and not (C % 16; for dφ nC % 16)
@pytest.mark.parametrize("B,n,C", [(4096, 4, 1024), (2000, 8, 520), (3000, 5, 1000)])
@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("unit", [0, 2])
def test_a_unit_without_its_copies(B, n, C, kernel, unit):
    c = case(B, n, C)
    assert mhc.mhc_device_status() == mhc.MHC_OK  # clears anything left over
    want = run(c, B, n, C, 5)
    assert mhc.mhc_device_status() == mhc.MHC_OK
    run(c, B, n, C, 5, (kernel, unit, 50_000_000))
    assert mhc.mhc_device_status() == mhc.MHC_ERR_TIMEOUT
    assert mhc.mhc_device_status() == mhc.MHC_OK  # reading cleared it
    again = run(c, B, n, C, 5)
    assert mhc.mhc_device_status() == mhc.MHC_OK
    for a, b in zip(want, again):
        assert torch.equal(a, b)


def test_the_hook_without_a_stall_is_the_call():
    B, n, C = 300, 4, 264
    c = case(B, n, C)
    for a, b in zip(run(c, B, n, C, 5), run(c, B, n, C, 5, (0, -1, 4_000_000_000))):
        assert torch.equal(a, b)
    assert mhc.mhc_device_status() == mhc.MHC_OK

"""The forward's steps back to back with everything between them filled with 0xFF first: a step starts while
the one before still runs, and has to wait for what it reads of it."""
import pytest
import torch

from gpu_util import cuda_ok
from test_train_gpu import ALPHA
from test_train_order_gpu import same_on_poison

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("n", range(1, 9))
@pytest.mark.parametrize("B,C,iters", [(1, 4096, 20), (700, 1024, 0), (20003, 256, 0), (9001, 1000, 20)])
def test_forward_steps_back_to_back(B, n, C, iters):
    K, N = n * C, n * n + 2 * n
    gen = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s, dtype=F32, std=1.0: (torch.randn(*s, device="cuda", generator=gen) * std).to(dtype)  # noqa: E731
    X, phi, F, bias = rnd(B, K, dtype=BF), rnd(N, K, std=K ** -0.5, dtype=BF), rnd(B, C, dtype=BF), rnd(N, std=0.3)
    o, again = mhc.alloc_outputs(B, n, C), mhc.alloc_outputs(B, n, C)
    H = [o["H_pre"], o["H_post"], o["H_res"]]

    def coeffs():
        mhc.mhc_coeffs(o["Y"], o["r"], *ALPHA, bias, iters, B, n, *H)

    def pre():
        mhc.mhc_pre_apply(X, o["H_pre"], B, n, C, o["F_pre"])

    def post():
        mhc.mhc_post_res_apply(X, F, o["H_res"], o["H_post"], B, n, C, o["X_next"])

    def fused():
        mhc.mhc_gemm_rms_coeffs(X, phi, *ALPHA, bias, iters, B, n, C, o["Y"], o["r"], *H, o["ws"])

    def following():  # the next layer on what post wrote
        mhc.mhc_gemm_rms_coeffs(o["X_next"], phi, *ALPHA, bias, iters, B, n, C, again["Y"], again["r"],
                                again["H_pre"], again["H_post"], again["H_res"], again["ws"])

    def step(*calls):
        def run():
            for c in calls:
                c()
        return run

    mhc.mhc_gemm_rms(X, phi, B, n, C, o["Y"], o["r"], o["ws"])
    same_on_poison(step(lambda: mhc.mhc_gemm_rms(X, phi, B, n, C, o["Y"], o["r"], o["ws"]), coeffs),
                   [o["Y"], o["r"], o["ws"]], H)
    same_on_poison(step(coeffs, pre), H, [o["F_pre"]])
    same_on_poison(step(coeffs, post), H, [o["X_next"]])
    same_on_poison(step(fused, pre, post), H + [o["ws"]], [o["F_pre"], o["X_next"]])
    same_on_poison(step(post, following), [o["X_next"], again["ws"]], [again["Y"], again["H_res"]])
    assert mhc.mhc_device_status() == mhc.MHC_OK


@pytest.mark.parametrize("n", range(1, 9))
@pytest.mark.parametrize("B,C", [(700, 1024), (20003, 256)])
def test_e4m3_steps_back_to_back(B, n, C):
    N = n * n + 2 * n
    gen = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    X, F = rnd(B, n * C).to(torch.float8_e4m3fn), rnd(B, C).to(torch.float8_e4m3fn)
    Y, r, bias = rnd(B, N), rnd(B).abs() + 0.5, rnd(N) * 0.3
    H = [torch.empty(B, n, device="cuda"), torch.empty(B, n, device="cuda"), torch.empty(B, n, n, device="cuda")]
    F_pre = torch.empty(B, C, dtype=torch.uint8, device="cuda")
    nxt = torch.empty(B, n * C, dtype=torch.uint8, device="cuda")

    def pre():
        mhc.mhc_coeffs(Y, r, *ALPHA, bias, 0, B, n, *H)
        mhc.mhc_pre_apply_e4m3(X, H[0], B, n, C, F_pre)

    def post():
        mhc.mhc_coeffs(Y, r, *ALPHA, bias, 0, B, n, *H)
        mhc.mhc_post_res_apply_e4m3(X, F, H[2], H[1], B, n, C, nxt)

    same_on_poison(pre, H, [F_pre])
    same_on_poison(post, H, [nxt])

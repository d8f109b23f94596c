"""What a kernel reads of the one before it: calls run back to back start while the kernel before still runs,
so everything in between (workspaces, kept codes, coefficients, gradients) is filled with 0xFF first, and the
outputs have to be those of the settled buffers, to the bit."""
import pytest
import torch

from gpu_util import cuda_ok
from test_train_gpu import ALPHA

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32 = torch.bfloat16, torch.float32


def same_on_poison(call, between, outs, turns=6):
    for _ in range(2):
        call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in want:
        assert bool(torch.isfinite(o.float()).all())
    for k in range(turns):
        for t in between:
            t.view(torch.uint8).fill_(0xFF)
        if k % 2:
            torch.cuda.synchronize()
        call()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), "output %d, turn %d" % (i, k)


SHAPES = [(20003, 1, 2504, 0), (20003, 1, 2504, 20), (60000, 1, 64, 1), (20003, 2, 1000, 0), (9000, 3, 1000, 1),
          (16000, 4, 1024, 0), (16000, 4, 1024, 20), (4001, 5, 520, 0), (4001, 6, 264, 1), (4001, 7, 200, 0),
          (4001, 8, 512, 0), (8191, 8, 256, 20), (20003, 8, 40, 60), (128, 4, 7168, 0), (1, 4, 7168, 20)]


@pytest.mark.parametrize("B,n,C,iters", SHAPES)
def test_training_calls_back_to_back(B, n, C, iters):
    K, N, V = n * C, n * n + 2 * n, 997
    gen = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s, dtype=F32, std=1.0: (torch.randn(*s, device="cuda", generator=gen) * std).to(dtype)  # noqa: E731
    e = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    table, ids = rnd(V, C, dtype=BF), torch.randint(0, V, (B,), device="cuda", generator=gen)
    phi, bias, F, G = rnd(N, K, std=K ** -0.5, dtype=BF), rnd(N, std=0.3), rnd(B, C, dtype=BF), rnd(B, n, C, std=1e-2, dtype=BF)
    X, nxt, back = (e(B, n, C, dtype=BF) for _ in range(3))
    o, (q, s) = mhc.alloc_outputs(B, n, C), mhc.alloc_kept(B, n, C)
    H = [o["H_pre"], o["H_post"], o["H_res"]]
    dF, dhr, dhq, dX = e(B, C, dtype=BF), e(B, n, n), e(B, n), e(B, n, C, dtype=BF)
    dphi, dbias, dalpha, dT = e(N, K), e(N), e(3), e(V, C)
    ws, wt = mhc.pre_backward_workspace(B, n, C, iters), mhc.embed_backward_workspace(V, B, n, C)

    def embed():
        mhc.mhc_embed(table, ids, 1.0, V, B, n, C, X)

    def coeffs():
        mhc.mhc_gemm_rms_coeffs(X, phi, *ALPHA, bias, iters, B, n, C, o["Y"], o["r"], *H, o["ws"])

    def keep():
        mhc.mhc_post_res_apply_ckpt(X, F, o["H_res"], o["H_post"], B, n, C, nxt, q, s)

    def post():
        mhc.mhc_post_res_apply_backward(G, q, s, F, o["H_post"], B, n, C, dF, dhr, dhq)

    def pre():
        mhc.mhc_pre_backward(G, dF, q, s, phi, *ALPHA, bias, iters, o["Y"], o["r"], *H, dhr, dhq, 0, B, n, C,
                             dX, dphi, dbias, dalpha, ws)

    def step(*calls):
        def run():
            for c in calls:
                c()
        return run

    embed()
    same_on_poison(step(embed, coeffs, keep), [X, o["Y"], o["r"], *H, o["ws"], q, s], [nxt, q, s])
    same_on_poison(step(keep, post), [q, s, nxt], [dF, dhr, dhq])
    same_on_poison(pre, [ws], [dX, dphi, dbias, dalpha])
    same_on_poison(step(keep, pre), [q, s, ws], [dX, dphi, dbias, dalpha])
    same_on_poison(step(post, pre), [dF, dhr, dhq, ws], [dX, dphi, dbias, dalpha])
    same_on_poison(step(pre, lambda: mhc.mhc_embed_backward(dX, ids, 1.0, 0, V, B, n, C, dT, wt)), [dX, ws, wt], [dT])
    same_on_poison(step(lambda: mhc.mhc_ckpt_pack(X, B, n, C, q, s), lambda: mhc.mhc_ckpt_unpack(q, s, B, n, C, back)),
                   [q, s], [back])
    assert mhc.mhc_device_status() == mhc.MHC_OK

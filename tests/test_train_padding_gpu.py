"""Tokens of zeros (padding ids) through the forward and the backward: r = 0, coefficients from the
bias, nothing added to the gradients of the weights."""
import math

import pytest
import torch

from gpu_util import cuda_ok
from test_train_gpu import ALPHA, normal, pre_case, pre_run
from train_util import MMA_STEP, U32, Guarded, coeffs64, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32 = torch.bfloat16, torch.float32
CALLS = ["mhc_forward", "mhc_testing_forward_chain", "mhc_testing_forward_decode", "mhc_testing_forward_fused",
         "mhc_gemm_rms_coeffs", "mhc_coeffs", "mhc_forward_f32w", "mhc_forward_e4m3"]


def forward(call, X, phi, F, bias, iters, B, n, C):
    o = mhc.alloc_outputs(B, n, C)
    X, F = X.reshape(B, n * C), F
    if call == "mhc_forward_f32w":
        split = torch.empty(2 * phi.shape[0], phi.shape[1], dtype=BF, device="cuda")
        mhc.mhc_split_phi(phi.float(), n, C, split)
        phi, F = split, F.float()
    if call == "mhc_forward_e4m3":
        X, phi, F = (t.float().to(torch.float8_e4m3fn) for t in (X, phi, F))
        o["F_pre"] = torch.empty(B, C, dtype=torch.uint8, device="cuda")
        o["X_next"] = torch.empty(B, n * C, dtype=torch.uint8, device="cuda")
    H = [o["H_pre"], o["H_post"], o["H_res"]]
    if call == "mhc_gemm_rms_coeffs":
        mhc.mhc_gemm_rms_coeffs(X, phi, *ALPHA, bias, iters, B, n, C, o["Y"], o["r"], *H, o["ws"])
    elif call == "mhc_coeffs":
        mhc.mhc_gemm_rms(X, phi, B, n, C, o["Y"], o["r"], o["ws"])
        mhc.mhc_coeffs(o["Y"], o["r"], *ALPHA, bias, iters, B, n, *H)
    else:
        getattr(mhc, call)(X, phi, F, *ALPHA, bias, iters, B, n, C, o["Y"], o["r"], *H, o["F_pre"],
                           o["X_next"], o["ws"])
    if call in ("mhc_gemm_rms_coeffs", "mhc_coeffs"):
        mhc.mhc_pre_apply(X, o["H_pre"], B, n, C, o["F_pre"])
        mhc.mhc_post_res_apply(X, F, o["H_res"], o["H_post"], B, n, C, o["X_next"])
    return o


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("n", [1, 4, 5, 8])
def test_forward_of_a_token_of_zeros(call, n):
    B, C, iters = 300, 16384 // n // 8 * 8 if "fused" in call else 1024, 20
    N = n * n + 2 * n
    X, phi = normal(1, B, n, C).cuda(), normal(2, N, n * C, std=0.05).cuda()
    F, bias = normal(3, B, C).cuda(), normal(4, N, std=0.5, dtype=F32).cuda()
    dead = [0, 127, 128, 299]
    whole = forward(call, X, phi, F, bias, iters, B, n, C)
    Z = X.clone()
    Z[dead] = 0
    o = forward(call, Z, phi, F, bias, iters, B, n, C)
    live = [b for b in range(B) if b not in dead]
    keys = ("Y", "r", "H_pre", "H_post", "H_res", "F_pre", "X_next")
    for k in keys:
        assert torch.equal(o[k][live], whole[k][live]), k  # the other tokens' bits
    assert not bool(o["r"][dead].any()) and not bool(o["Y"][dead].any())
    hp, hq, hr = coeffs64(torch.zeros(1, N, dtype=torch.float64), torch.ones(1, dtype=torch.float64), ALPHA,
                          bias.double().cpu(), iters, n)
    # exp, a sum, a reciprocal within an ulp; Sinkhorn: 2·iters steps of n + 3 such roundings
    for k, ref, steps in (("H_pre", hp, 8), ("H_post", hq, 8), ("H_res", hr, 2 * iters * (n + 3) + 8)):
        within(o[k][dead], ref.expand(len(dead), *ref.shape[1:]), steps * U32 * 2, k)
    assert not bool((o["F_pre"][dead].view(torch.uint8) & 127).any())
    if call != "mhc_forward_e4m3":  # X_next = H_post ⊗ F_out
        want = (o["H_post"][dead][:, :, None] * F[dead].float()[:, None, :]).to(BF).view(len(dead), n * C)
        assert torch.equal(o["X_next"][dead], want)


PADS = [(24, 1, 72), (40, 4, 136), (56, 5, 96), (33, 8, 264)]


def grown(d, B, total, n, C, gradient):
    """The case with tokens of zeros behind its own, up to `total`."""
    p, more = dict(d), total - B
    zeros = dict(q=0, s=10, Y=0.0, r=0.0, G=0.0, dF=0.0, dhr=0.0, dhq=0.0)
    N = n * n + 2 * n
    hp, hq, hr = coeffs64(torch.zeros(more, N, dtype=torch.float64), torch.ones(more, dtype=torch.float64),
                          ALPHA, d["bias"].double(), 20, n)
    for k in ("q", "s", "Y", "r", "G", "dF", "dhr", "dhq"):
        p[k] = torch.cat([d[k], torch.full((more, *d[k].shape[1:]), zeros[k], dtype=d[k].dtype)])
    p["hp"], p["hq"], p["hr"] = (torch.cat([d[k], h.float()]) for k, h in (("hp", hp), ("hq", hq), ("hr", hr)))
    if gradient:
        p["G"][B:], p["dF"][B:] = normal(5, more, n, C, std=1e-2), normal(6, more, C, std=1e-2)
        p["dhr"][B:], p["dhq"][B:] = normal(7, more, n, n, std=0.1, dtype=F32), normal(8, more, n, std=0.1, dtype=F32)
    return p


@pytest.mark.parametrize("B,n,C", PADS)
def test_padding_adds_nothing(B, n, C):
    """Behind the batch, within its block of 64 tokens, so that the sums run in the same order."""
    d = pre_case(B + n, B, n, C, 20)
    want, _ = pre_run(d, B, n, C, 20, Guarded())
    out, _ = pre_run(grown(d, B, B + 5, n, C, False), B + 5, n, C, 20, Guarded())
    for k in ("dphi", "dbias", "dalpha"):
        assert bool(torch.isfinite(out[k]).all()), k
        assert torch.equal(out[k], want[k]), k
    assert torch.equal(out["dX"][:B], want["dX"]) and not bool(out["dX"][B:].any())


@pytest.mark.parametrize("B,n,C", PADS)
def test_a_gradient_that_comes_in_for_padding(B, n, C):
    """It reaches the bias alone; that token's dX has no value, every other result is what it was."""
    d = pre_case(B + n, B, n, C, 20)
    want, _ = pre_run(d, B, n, C, 20, Guarded())
    out, _ = pre_run(grown(d, B, B + 5, n, C, True), B + 5, n, C, 20, Guarded())
    for k in ("dphi", "dalpha"):
        assert torch.equal(out[k], want[k]), k
    assert bool(torch.isfinite(out["dbias"]).all()) and not torch.equal(out["dbias"], want["dbias"])
    assert torch.equal(out["dX"][:B], want["dX"])
    assert bool(torch.isnan(out["dX"][B:]).all())


def test_a_batch_with_padding_ids():
    """Ids to the loss's gradient and back over two layers: padding between the tokens, which the loss
    leaves out, changes no gradient but in its rounding."""
    B, n, C, iters, V = 60, 4, 136, 20, 30
    N, K, scale = n * n + 2 * n, n * C, math.sqrt(C)
    table = normal(1, V, C, std=0.05, dtype=F32).cuda()
    phi = [normal(2 + k, N, K, std=0.05).cuda() for k in (0, 1)]
    bias = [normal(4 + k, N, std=0.5, dtype=F32).cuda() for k in (0, 1)]
    W = [normal(6 + k, C, C, std=C ** -0.5).cuda().float() for k in (0, 1)]
    gen = torch.Generator().manual_seed(8)
    live_ids = torch.randint(0, V, (B,), generator=gen)
    last = normal(9, B, n, C, std=1e-2)
    at = torch.arange(B) + torch.arange(B) // 4  # a padding id after each fourth token

    def step(ids, dX):
        b = len(ids)
        e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        X, kept = e(b, n, C, dtype=BF), []
        mhc.mhc_embed_f32(table, ids.cuda(), scale, V, b, n, C, X)
        for k in (0, 1):
            o, q = mhc.alloc_outputs(b, n, C), mhc.alloc_kept(b, n, C)
            mhc.mhc_gemm_rms_coeffs(X, phi[k], *ALPHA, bias[k], iters, b, n, C, o["Y"], o["r"], o["H_pre"],
                                    o["H_post"], o["H_res"], o["ws"])
            mhc.mhc_pre_apply(X, o["H_pre"], b, n, C, o["F_pre"])
            F = (torch.tanh(o["F_pre"].float()) @ W[k]).to(BF)
            nxt = e(b, n, C, dtype=BF)
            mhc.mhc_post_res_apply_ckpt(X, F, o["H_res"], o["H_post"], b, n, C, nxt, *q)
            kept.append((o, q, F))
            X = nxt
        grads, dX = {}, dX.cuda()
        for k in (1, 0):
            o, q, F = kept[k]
            dF, dhr, dhq = e(b, C, dtype=BF), e(b, n, n), e(b, n)
            mhc.mhc_post_res_apply_backward(dX, *q, F, o["H_post"], b, n, C, dF, dhr, dhq)
            t = torch.tanh(o["F_pre"].float())
            grads["W%d" % k] = t.t() @ dF.float()
            dF_pre = ((dF.float() @ W[k].t()) * (1 - t * t)).to(BF)
            dphi, dbias, dalpha = e(N, K), e(N), e(3)
            mhc.mhc_pre_backward(dX, dF_pre, *q, phi[k], *ALPHA, bias[k], iters, o["Y"], o["r"], o["H_pre"],
                                 o["H_post"], o["H_res"], dhr, dhq, 0, b, n, C, dX, dphi, dbias, dalpha,
                                 mhc.pre_backward_workspace(b, n, C, iters))
            grads.update({"phi%d" % k: dphi, "bias%d" % k: dbias, "alpha%d" % k: dalpha})
        dT = e(V, C)
        mhc.mhc_embed_backward(dX, ids.cuda(), scale, 0, V, b, n, C, dT, mhc.embed_backward_workspace(V, b, n, C))
        grads["table"] = dT
        return grads

    want = step(live_ids, last)
    total = int(at[-1]) + 1
    ids, dX = torch.full((total,), -1), torch.zeros(total, n, C, dtype=BF)
    ids[at], dX[at] = live_ids, last
    assert int((ids < 0).sum()) >= 14
    got = step(ids, dX)
    for k, w in want.items():
        assert bool(torch.isfinite(got[k]).all()), k
        # the same terms, at most 60, in another order: two chains of about 100 additions (the
        # tensor cores' drop 2^-19 a step) of partial sums that stay under 16 times the largest result
        off = float((got[k].double() - w.double()).abs().max())
        assert off <= 16 * (200 * U32 + 2 * 16 * MMA_STEP) * float(w.abs().max()), (k, off)

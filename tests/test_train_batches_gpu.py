"""Batches that the training kernels walk: several units of work a CTA (rings that wrap, token tiles, strips
and accumulation chains that end inside a CTA), the forms taken once there is a warp a token, coefficients
of more tokens than one walk, more rows than a grid's y.  Every output against 64 bits, computed on the GPU."""
import pytest
import torch

from gpu_util import cuda_ok
from test_train_gpu import ALPHA
from train_util import HALF_BF16, MMA_STEP, U32, pack64, sinkhorn64, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def past_a_warp_a_token():
    """Just above the batch from which a warp takes a token, and no multiple of a CTA's eight."""
    return 16 * sms() + 5


class Rand:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)

    def __call__(self, *s, std=1.0, dtype=F32):
        return (torch.randn(*s, device="cuda", generator=self.gen) * std).to(dtype)


def unset(*s, dtype=F32):
    return torch.full(s, float("nan"), dtype=dtype, device="cuda")


def kept(X):
    """(codes, scales, the values they stand for in 64 bits)"""
    B, n, C = X.shape
    q, s = mhc.alloc_kept(B, n, C)
    mhc.mhc_ckpt_pack(X, B, n, C, q, s)
    x = q.view(torch.float8_e4m3fn).double()
    return q, s, x * torch.exp2(s.double() - 127).repeat_interleave(32, -1)[..., :C]


def check(got, ref, tol, what):
    off = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all()), "%s: not finite" % what
    bad = off > tol
    assert not bool(bad.any()), "%s: %d of %d values outside, the worst by %.3e" % (
        what, int(bad.sum()), bad.numel(), float((off - tol).max()))


# ----------------------------------------------------- backward of the update


@pytest.mark.parametrize("ft", [BF, F32])
@pytest.mark.parametrize("n", range(1, 9))
@pytest.mark.parametrize("B,C", [(None, 72), (None, 520), (7, 264), (1, 1000)])
def test_post_res_apply_backward(B, n, C, ft):
    B = B or past_a_warp_a_token()
    rnd = Rand(n * C + B)
    q, s, x = kept(rnd(B, n, C, dtype=BF) * rnd(B, 1, 1).exp().to(BF))
    G, F, hq = rnd(B, n, C, std=1e-2, dtype=BF), rnd(B, C, dtype=ft), 2 * torch.sigmoid(rnd(B, n))
    dF, dhr, dhq = unset(B, C, dtype=ft), unset(B, n, n), unset(B, n)
    f = mhc.mhc_post_res_apply_backward if ft == BF else mhc.mhc_post_res_apply_backward_f32
    f(G, q, s, F, hq, B, n, C, dF, dhr, dhq)
    g, h = G.double(), hq.double()
    ref, terms = torch.einsum("bi,bic->bc", h, g), torch.einsum("bi,bic->bc", h, g.abs())
    # n <= 4: fp32 multiply-adds, a lane's every 256th or 2048th group of 8 channels in pairs, then
    # the two of a pair, five shuffles and up to eight warps.  n >= 5: tensor-core products of a block,
    # three terms of H_post
    chain = (C / 64 + 24) * U32
    off = (n + 3) * U32 if n < 5 else 2 * MMA_STEP + 2.0 ** -25
    check(dF, ref, (HALF_BF16 if ft == BF else U32) * ref.abs() + 1.01 * off * terms, "dF_out")
    terms = g.abs() @ x.abs().transpose(1, 2)
    check(dhr, g @ x.transpose(1, 2), (chain if n < 5 else 2 * MMA_STEP + chain) * terms, "dH_res")
    terms = torch.einsum("bic,bc->bi", g.abs(), F.double().abs())
    off = chain if n < 5 or ft == F32 else 2 * MMA_STEP + chain
    check(dhq, torch.einsum("bic,bc->bi", g, F.double()), off * terms, "dH_post")


# ------------------------------------------------ backward of steps 1 to 4a

PRE = [
    # tokens, n, C, steps: what a CTA of dX (64 tokens x 64 or 32 channels a unit) and of dφ (256
    # channels x 64 tokens) goes through
    (20000, 4, 72, 3),     # tiles change; codes not by TMA in dX; scales byte by byte
    (20000, 4, 128, 20),   # tiles change; scales in words
    (20000, 5, 72, 5),     # codes not by TMA in either
    (2440, 8, 1000, 20),   # many chunks a tile, codes not by TMA in dX, scales in words
    (2440, 8, 256, 20),
    (5000, 8, 160, 7),     # scales byte by byte
    (20003, 4, 600, 1),    # chains of 16 blocks, strips that end inside a CTA
    (20003, 1, 2504, 20),  # the same, codes not by TMA in dφ
    (20003, 8, 304, 2),    # the same, n = 8
    (9001, 7, 200, 0),     # no step at all, codes not by TMA in either
]
# and without a step, where the sums over tokens are known to a few roundings of each token's share
PRE += [(B, n, C, 0) for B, n, C, iters in PRE if iters]
PRE += [(None, n, C, 20) for n in range(1, 9) for C in (40, 264)]  # a warp a token in the dH_pre sums
# the coefficients' loop goes round twice: its history in shared memory, and in the workspace
PRE += [(160001, 4, 8, 3), (160001, 8, 8, 2), (20003, 4, 8, 60), (20003, 8, 8, 60)]


@pytest.mark.parametrize("B,n,C,iters", PRE)
def test_pre_backward(B, n, C, iters):
    B = B or past_a_warp_a_token()
    K, N = n * C, n * n + 2 * n
    rnd = Rand(B + 3 * n + C)
    q, s, x = kept(rnd(B, n, C, dtype=BF) * rnd(B, 1, 1).exp().to(BF))
    phi, bias = rnd(N, K, std=K ** -0.5, dtype=BF), rnd(N, std=0.5)
    xk = x.view(B, K)
    Y, r = (xk @ phi.double().t()).float(), xk.square().mean(1).sqrt().float()
    al = torch.tensor([ALPHA[0]] * n + [ALPHA[1]] * n + [ALPHA[2]] * n * n, dtype=F64, device="cuda")
    Ht = al * Y.double() / r.double()[:, None] + bias.double()
    hp, hq = torch.sigmoid(Ht[:, :n]).float(), (2 * torch.sigmoid(Ht[:, n:2 * n])).float()
    hr = sinkhorn64(Ht[:, 2 * n:].view(B, n, n), iters).float().contiguous()
    G, dF = rnd(B, n, C, std=1e-2, dtype=BF), rnd(B, C, std=1e-2, dtype=BF)
    dhr, dhq = rnd(B, n, n, std=0.1), rnd(B, n, std=0.1)
    ws = mhc.pre_backward_workspace(B, n, C, iters)

    def call():
        out = dict(dX=unset(B, n, C, dtype=BF), dphi=unset(N, K), dbias=unset(N), dalpha=unset(3))
        mhc.mhc_pre_backward(G, dF, q, s, phi, *ALPHA, bias, iters, Y, r, hp, hq, hr, dhr, dhq, 0, B, n, C,
                             out["dX"], out["dphi"], out["dbias"], out["dalpha"], ws)
        return out

    out, again = call(), call()
    assert mhc.mhc_device_status() == mhc.MHC_OK
    for k in out:
        assert torch.equal(out[k], again[k]), k

    Y, r, phi, hp, hq, hr, dhr, dhq, g, df = (t.double() for t in (Y, r, phi, hp, hq, hr, dhr, dhq, G, dF))
    H = Ht[:, 2 * n:].reshape(B, n, n).requires_grad_(True)
    with torch.enable_grad():
        P = sinkhorn64(H, iters)
        dres = torch.autograd.grad(P, H, dhr)[0].reshape(B, n * n)
    H, P = H.detach(), P.detach()
    dhp, dhp_t = torch.einsum("bc,bic->bi", df, x), torch.einsum("bc,bic->bi", df.abs(), x.abs())
    dHt = torch.cat([dhp * hp * (1 - hp), dhq * hq * (1 - hq / 2), dres], 1)
    t_pre = (C / 32 + 60) * U32 * dhp_t * hp * (1 - hp) + 4 * U32 * dhp.abs() * hp
    if iters:  # as in test_train_gpu.py
        size = (dhr.abs() * P.clamp_min(1.0)).sum((1, 2)) * (1 + H.abs().amax((1, 2)))
        t_res = (4 * iters + 4) * (n + 8) * U32 * size[:, None].expand(B, n * n)
    else:  # H̃ in four roundings, exp within two units of the last place, a product
        h = H.view(B, n * n)
        t_res = (4 * ((h - bias[2 * n:].double()).abs() + h.abs()) + 6) * U32 * dres.abs()
    t_H = torch.cat([t_pre, 6 * U32 * (dhq * hq).abs(), t_res], 1)
    dY, t_Y = al * dHt / r[:, None], al * t_H / r[:, None]
    t_Y = t_Y + 4 * U32 * dY.abs()
    # sums over tokens: 64 a CTA and turn in four chains, then the CTAs
    steps = B / 64 / 32 + 60
    check(out["dbias"], dHt.sum(0), t_H.sum(0) + steps * U32 * dHt.abs().sum(0), "dbias")
    yr = Y / r[:, None]
    each, t_each = (dHt * yr).sum(0), ((t_H + (steps + n * n) * U32 * dHt.abs()) * yr.abs()).sum(0)
    cut = lambda t: torch.stack([v.sum() for v in t.split([n, n, n * n])])  # noqa: E731
    check(out["dalpha"], cut(each), cut(t_each), "dalpha")
    # three bf16 terms leave 2^-25 of dY; chains of 64 tensor-core steps, joined by additions
    off = 64 * MMA_STEP + 2.0 ** -25 + (B / 1024 + 40) * U32
    check(out["dphi"], dY.t() @ xk, t_Y.t() @ xk.abs() + off * (dY.abs().t() @ xk.abs()), "dphi")
    sx = -(dY * Y).sum(1) / (K * r * r)
    t_sx = (((t_Y + (N + 8) * U32 * dY.abs()) * Y.abs()).sum(1)) / (K * r * r)
    ref = hr.transpose(1, 2) @ g + hp[:, :, None] * df[:, None, :] + (dY @ phi).view(B, n, C)
    ref += sx[:, None, None] * x
    t_proj = (dY.abs() @ phi.abs()).view(B, n, C)
    tol = (hr.transpose(1, 2) @ g.abs() + (hp[:, :, None] * df[:, None, :]).abs() + t_proj +
           (sx[:, None, None] * x).abs()) * (n + 6) * U32
    # dY as two bf16 terms
    tol += HALF_BF16 * ref.abs() + t_sx[:, None, None] * x.abs() + 1.01 * (t_Y @ phi.abs()).view(B, n, C)
    tol += 1.01 * (2.0 ** -16 + 2 * ((N + 15) // 16) * MMA_STEP) * t_proj
    check(out["dX"], ref, tol, "dX")


# ------------------------------------------------------------------- 8 bits


def test_pack_more_rows_than_a_grid_has():
    B, n, C = 66000, 4, 8  # four rows a thread, 65535 of them at most in y
    X = Rand(1)(B, n, C, dtype=BF)
    q, s, _ = kept(X)
    rq, rs = pack64(X)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)
    back = unset(B, n, C, dtype=BF)
    mhc.mhc_ckpt_unpack(q, s, B, n, C, back)
    within(back, X.double().cpu(), 2.0 ** -4 * X.double().cpu().abs() + 2.0 ** -10 *
           torch.exp2(rs.double() - 127), "X as kept")

"""The training operators on the GPU against their formulas in 64 bits (train_util)."""
import math

import pytest
import torch

from gpu_util import cuda_ok
from train_util import (HALF_BF16, MMA_STEP, U32, Guarded, coeffs64, layer64, pack64, sinkhorn64,
                        unpack64, within)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1, 8), (1, 4, 7168), (3, 2, 40), (9, 3, 72), (33, 4, 264), (65, 4, 1000), (7, 5, 264),
          (5, 6, 96), (66, 7, 72), (130, 8, 136), (2, 8, 1000)]


def normal(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(dtype)


def streams(seed, B, n, C):
    """X with tokens of very different size, and blocks that are zero or tiny."""
    X = normal(seed, B, n, C, dtype=torch.float64)
    X *= 10.0 ** (2 * torch.rand(B, 1, 1, generator=torch.Generator().manual_seed(seed + 1),
                                 dtype=torch.float64) - 1)
    if C > 64 and B > 2:
        X[1, 0, 32:64] = 0
        X[2, n - 1, :32] *= 1e-30
    return X.to(BF)


# --------------------------------------------------------------- X in 8 bits


@pytest.mark.parametrize("B,n,C", SHAPES)
def test_pack_and_unpack(B, n, C):
    X = streams(B + n + C, B, n, C)
    g = Guarded()
    Xd, q, s = g.put(X), g.empty(B, n, C, dtype=torch.uint8), g.empty(B, n, -(-C // 32), dtype=torch.uint8)
    back = g.empty(B, n, C, dtype=BF)
    mhc.mhc_ckpt_pack(Xd, B, n, C, q, s)
    mhc.mhc_ckpt_unpack(q, s, B, n, C, back)
    torch.cuda.synchronize()
    g.check()
    rq, rs = pack64(X)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq)
    assert torch.equal(back.double().cpu(), unpack64(rq, rs))


def test_pack_at_the_borders_of_the_format():
    """Largest magnitudes around 448·2^k, the ends of bf16's range, signed zeros, ties."""
    rows = []
    for top in (448.0, 450.0, 1.75, 1.7578125, 1.0, 3.3895e38, 2.0 ** 127, 2.0 ** -126, 2.0 ** -133,
                2.0 ** -109, 448 * 2.0 ** -117, 450 * 2.0 ** -117, 0.0):
        row = torch.zeros(32, dtype=torch.float64)
        row[0] = top
        row[1] = -top
        row[2:30] = top * torch.linspace(-1, 1, 28, dtype=torch.float64)
        row[30], row[31] = -0.0, top * 2.0 ** -16
        rows.append(row)
    ties = torch.arange(32, dtype=torch.float64) * 0.5 + 240.0  # halves of e4m3 steps under 448
    rows += [ties, -ties, ties * 2.0 ** -14]
    rows[-1][0] = 448.0
    X = torch.stack(rows).to(BF).view(len(rows), 1, 32)
    B = len(rows)
    q = torch.empty(B, 1, 32, dtype=torch.uint8, device="cuda")
    s = torch.empty(B, 1, 1, dtype=torch.uint8, device="cuda")
    mhc.mhc_ckpt_pack(X.cuda(), B, 1, 32, q, s)
    rq, rs = pack64(X)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq)
    back = torch.empty(B, 1, 32, dtype=BF, device="cuda")
    mhc.mhc_ckpt_unpack(q, s, B, 1, 32, back)
    assert torch.equal(back.double().cpu(), unpack64(rq, rs))


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_block_that_is_not_finite_is_kept_as_nan_alone(bad):
    B, n, C = 3, 2, 72
    X = streams(5, B, n, C)
    X[1, 1, 40] = bad
    q, s = mhc.alloc_kept(B, n, C)
    back = torch.empty(B, n, C, dtype=BF, device="cuda")
    mhc.mhc_ckpt_pack(X.cuda(), B, n, C, q, s)
    mhc.mhc_ckpt_unpack(q, s, B, n, C, back)
    nan = torch.isnan(back.cpu())
    assert bool(nan[1, 1, 32:64].all()) and int(nan.sum()) == 32
    assert int(s[1, 1, 1]) == 255


def coefs(seed, B, n):
    H_res = sinkhorn64(normal(seed, B, n, n, std=0.5, dtype=torch.float64), 20).float()
    return H_res, (2 * torch.sigmoid(normal(seed + 1, B, n, dtype=torch.float64))).float()


@pytest.mark.parametrize("ft", [BF, F32])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,n,C", SHAPES)
def test_post_res_apply_ckpt(B, n, C, in_place, ft):
    X, F = streams(3 * B + n, B, n, C), normal(2, B, C, dtype=ft)
    H_res, H_post = coefs(7, B, n)
    g = Guarded()
    Xd = g.put(X)
    nxt = Xd if in_place else g.empty(B, n, C, dtype=BF)
    q, s = g.empty(B, n, C, dtype=torch.uint8), g.empty(B, n, -(-C // 32), dtype=torch.uint8)
    f = mhc.mhc_post_res_apply_ckpt if ft == BF else mhc.mhc_post_res_apply_ckpt_f32
    f(Xd, g.put(F), g.put(H_res), g.put(H_post), B, n, C, nxt, q, s)
    torch.cuda.synchronize()
    g.check()
    rq, rs = pack64(X)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)
    x, h, hq = X.double(), H_res.double(), H_post.double()[:, :, None]
    ref = h @ x + hq * F.double()[:, None, :]
    terms = h.abs() @ x.abs() + (hq * F.double()[:, None, :]).abs()
    within(nxt, ref, HALF_BF16 * ref.abs() + 1.01 * (n + 2) * U32 * terms, "X_next")


# ----------------------------------------------------- backward of the update


def post_case(seed, B, n, C, ft):
    q, s = pack64(streams(seed, B, n, C))
    return dict(G=normal(seed + 1, B, n, C, std=1e-2), q=q, s=s, F=normal(seed + 2, B, C, dtype=ft),
                H_post=coefs(seed + 3, B, n)[1])


def post_run(d, B, n, C, ft, g):
    out = dict(dF=g.empty(B, C, dtype=ft), dH_res=g.empty(B, n, n), dH_post=g.empty(B, n))
    f = mhc.mhc_post_res_apply_backward if ft == BF else mhc.mhc_post_res_apply_backward_f32
    f(g.put(d["G"]), g.put(d["q"]), g.put(d["s"]), g.put(d["F"]), g.put(d["H_post"]), B, n, C,
      out["dF"], out["dH_res"], out["dH_post"])
    return out


@pytest.mark.parametrize("ft", [BF, F32])
@pytest.mark.parametrize("B,n,C", SHAPES)
def test_post_res_apply_backward(B, n, C, ft):
    d = post_case(B * n + C, B, n, C, ft)
    g = Guarded()
    out = post_run(d, B, n, C, ft, g)
    torch.cuda.synchronize()
    g.check()
    x, G, F, hq = unpack64(d["q"], d["s"]), d["G"].double(), d["F"].double(), d["H_post"].double()
    ref = torch.einsum("bi,bic->bc", hq, G)
    terms = torch.einsum("bi,bic->bc", hq, G.abs())
    half = HALF_BF16 if ft == BF else U32
    # n >= 5: tensor-core products of three bf16 terms of H_post, in two steps
    off = (n + 3) * U32 if n < 5 else 2 * MMA_STEP + 2.0 ** -25
    within(out["dF"], ref, half * ref.abs() + 1.01 * off * terms, "dF_out")
    terms = G.abs() @ x.abs().transpose(1, 2)
    within(out["dH_res"], G @ x.transpose(1, 2), (MMA_STEP * (C / 16 + 2) + 32 * U32) * terms, "dH_res")
    terms = torch.einsum("bic,bc->bi", G.abs(), F.abs())
    off = (C / 4 + 40) * U32 if n < 5 or ft == F32 else 2 * MMA_STEP + (C / 32 + 40) * U32
    within(out["dH_post"], torch.einsum("bic,bc->bi", G, F), off * terms, "dH_post")


def test_a_kept_nan_stays_in_its_token():
    B, n, C = 6, 4, 264
    d = post_case(11, B, n, C, BF)
    clean = post_run(d, B, n, C, BF, Guarded())
    d["s"][2, 1, 3], d["q"][2, 1, 96:128] = 255, 127
    out = post_run(d, B, n, C, BF, Guarded())
    assert torch.equal(out["dF"], clean["dF"]) and torch.equal(out["dH_post"], clean["dH_post"])
    nan = torch.isnan(out["dH_res"].cpu())
    assert bool(nan[2, :, 1].all()) and int(nan.sum()) == n
    keep = ~nan
    assert torch.equal(out["dH_res"].cpu()[keep], clean["dH_res"].cpu()[keep])


# ------------------------------------------------ backward of steps 1 to 4a

ALPHA = (0.05, 0.07, 0.11)


def pre_case(seed, B, n, C, iters):
    K, N = n * C, n * n + 2 * n
    X = streams(seed, B, n, C)
    q, s = pack64(X)
    phi_t, bias = normal(seed + 1, N, K, std=0.05), normal(seed + 2, N, std=0.5, dtype=F32)
    x = X.double().view(B, K)
    Y, r = (x @ phi_t.double().t()).float(), x.square().mean(1).sqrt().float()
    hp, hq, hr = coeffs64(Y.double(), r.double(), ALPHA, bias.double(), iters, n)
    return dict(G=normal(seed + 3, B, n, C, std=1e-2), dF=normal(seed + 4, B, C, std=1e-2), q=q, s=s,
                phi=phi_t, bias=bias, Y=Y, r=r, hp=hp.float(), hq=hq.float(), hr=hr.float(),
                dhr=normal(seed + 5, B, n, n, std=0.1, dtype=F32),
                dhq=normal(seed + 6, B, n, std=0.1, dtype=F32))


def pre_run(d, B, n, C, iters, g, accumulate=0, start=None, in_place=False, stream=None):
    K, N = n * C, n * n + 2 * n
    G = g.put(d["G"])
    out = dict(dX=G if in_place else g.empty(B, n, C, dtype=BF), dphi=g.empty(N, K), dbias=g.empty(N),
               dalpha=g.empty(3))
    for k, v in (start or {}).items():
        out[k].copy_(v)
    ws = g.empty(mhc.pre_backward_workspace(B, n, C, iters).numel(), dtype=torch.uint8)
    args = [g.put(d[k]) for k in ("Y", "r", "hp", "hq", "hr", "dhr", "dhq")]
    call = lambda: mhc.mhc_pre_backward(G, args_in[0], args_in[1], args_in[2], args_in[3], *ALPHA,  # noqa: E731
                                        args_in[4], iters, *args, accumulate, B, n, C, out["dX"],
                                        out["dphi"], out["dbias"], out["dalpha"], ws, stream)
    args_in = [g.put(d[k]) for k in ("dF", "q", "s", "phi", "bias")]
    call()
    return out, call


def pre_ref(d, B, n, C, iters):
    """The gradients in 64 bits and, for each, what fp32 arithmetic may be off by."""
    K, N = n * C, n * n + 2 * n
    f = {k: v.double() for k, v in d.items() if k not in ("q", "s")}
    x = unpack64(d["q"], d["s"])
    Y, r, phi = f["Y"], f["r"], f["phi"]
    al = torch.tensor([ALPHA[0]] * n + [ALPHA[1]] * n + [ALPHA[2]] * n * n, dtype=torch.float64)
    Ht = (al * Y / r[:, None] + f["bias"])[:, 2 * n:].reshape(B, n, n).requires_grad_(True)
    P = sinkhorn64(Ht, iters)
    dres = torch.autograd.grad(P, Ht, f["dhr"])[0]
    dhp = torch.einsum("bc,bic->bi", f["dF"], x)
    dHt = torch.cat([dhp * f["hp"] * (1 - f["hp"]), f["dhq"] * f["hq"] * (1 - f["hq"] / 2),
                     dres.reshape(B, n * n)], 1)
    # dH_pre: a chain of C/4 + 40 additions; the sigmoid's three products
    dhp_t = torch.einsum("bc,bic->bi", f["dF"].abs(), x.abs())
    t_pre = (C / 4 + 50) * U32 * dhp_t * f["hp"] * (1 - f["hp"]) + 4 * U32 * dhp.abs() * f["hp"]
    t_post = 6 * U32 * (f["dhq"] * f["hq"]).abs()
    # Sinkhorn: 2·iters steps there and back, each n + 8 roundings of values that the
    # entries of the iterate (at most 1, or exp(H̃) without a step) weigh; H̃ itself is
    # off by a few roundings, which changes the iterate by as much
    size = (f["dhr"].abs() * P.detach().clamp_min(1.0 if iters else 0.0)).sum((1, 2))
    size = size * (1 + Ht.detach().abs().amax((1, 2)))
    t_res = (4 * iters + 4) * (n + 8) * U32 * size[:, None].expand(B, n * n)
    t_H = torch.cat([t_pre, t_post, t_res], 1)
    yr = Y / r[:, None]
    dY, t_Y = al * dHt / r[:, None], al * t_H / r[:, None]
    t_Y = t_Y + 4 * U32 * dY.abs()
    sx = -(dY * Y).sum(1) / (K * r * r)
    t_sx = (((t_Y + (N + 8) * U32 * dY.abs()) * Y.abs()).sum(1)) / (K * r * r)
    ref, tol = {}, {}
    ref["dbias"] = dHt.sum(0)
    tol["dbias"] = t_H.sum(0) + (B / 32 + 40) * U32 * dHt.abs().sum(0)
    each, t_each = (dHt * yr).sum(0), ((t_H + (B / 16 + n * n + 50) * U32 * dHt.abs()) * yr.abs()).sum(0)
    cut = [n, n, n * n]
    ref["dalpha"] = torch.stack([v.sum() for v in each.split(cut)])
    tol["dalpha"] = torch.stack([v.sum() for v in t_each.split(cut)])
    xk = x.view(B, K)
    ref["dphi"] = dY.t() @ xk
    # three bf16 terms leave 2^-25 of dY; B/16 + 8 tensor-core steps of three terms each
    tol["dphi"] = t_Y.t() @ xk.abs() + (3 * MMA_STEP * (B / 16 + 8) + 2.0 ** -25) * (dY.abs().t() @ xk.abs())
    proj = (dY @ phi).view(B, n, C)
    t_proj = dY.abs() @ phi.abs()
    mix = f["hr"].transpose(1, 2) @ f["G"]
    ref["dX"] = mix + f["hp"][:, :, None] * f["dF"][:, None, :] + proj + sx[:, None, None] * x
    terms = (f["hr"].transpose(1, 2) @ f["G"].abs() + (f["hp"][:, :, None] * f["dF"][:, None, :]).abs() +
             t_proj.view(B, n, C) + (sx[:, None, None] * x).abs())
    # dY enters this product as one bf16
    tol["dX"] = (HALF_BF16 * ref["dX"].abs() + (n + 6) * U32 * terms + t_sx[:, None, None] * x.abs() +
                 ((HALF_BF16 + MMA_STEP * (N / 16 + 1)) * t_proj + t_Y @ phi.abs()).view(B, n, C) * 1.01)
    return ref, tol


PRE = [(B, n, C, it) for (B, n, C), it in zip(SHAPES, (20, 20, 1, 5, 20, 3, 20, 0, 20, 20, 7))] + [
    (1, 8, 8, 20), (64, 4, 32, 0), (200, 1, 64, 20), (129, 2, 2056, 2)]


@pytest.mark.parametrize("B,n,C,iters", PRE)
def test_pre_backward(B, n, C, iters):
    d = pre_case(B + 3 * n + C, B, n, C, iters)
    g = Guarded()
    out, _ = pre_run(d, B, n, C, iters, g)
    torch.cuda.synchronize()
    g.check()
    assert mhc.mhc_device_status() == mhc.MHC_OK
    ref, tol = pre_ref(d, B, n, C, iters)
    for k in ("dbias", "dalpha", "dphi", "dX"):
        within(out[k], ref[k], tol[k], k)


@pytest.mark.parametrize("term", ["G", "dF", "phi", "X"])
@pytest.mark.parametrize("B,n,C", [(70, 1, 200), (130, 2, 72), (65, 3, 264), (200, 4, 136), (70, 4, 2056),
                                   (67, 5, 96), (66, 6, 264), (131, 7, 72), (129, 8, 136), (70, 8, 288)])
def test_each_term_of_dX_alone(B, n, C, term):
    """The other terms' inputs are zero, so that an error in a small term is not hidden by a large one's
    rounding (H̃ does not depend on X where Y is zero)."""
    d = pre_case(B + n, B, n, C, 5)
    zero = {"G": ("dF", "dhr", "dhq"), "dF": ("G", "phi", "dhr", "dhq", "Y"), "phi": ("G", "dF", "Y"),
            "X": ("G", "dF", "phi")}[term]
    for k in zero:
        d[k] = torch.zeros_like(d[k])
    out, _ = pre_run(d, B, n, C, 5, Guarded())
    ref, tol = pre_ref(d, B, n, C, 5)
    assert float(ref["dX"].abs().max()) > 0
    within(out["dX"], ref["dX"], tol["dX"], "dX")


def test_pre_backward_many_iterations_keep_their_history_in_the_workspace():
    """More steps than shared memory holds (2·8·64·4 bytes each), and more tokens than one walk."""
    B, n, C, iters = 300, 8, 40, 60
    d = pre_case(3, B, n, C, iters)
    out, _ = pre_run(d, B, n, C, iters, Guarded())
    ref, tol = pre_ref(d, B, n, C, iters)
    for k in ref:
        within(out[k], ref[k], tol[k], k)


def test_pre_backward_in_place_and_repeated():
    B, n, C, iters = 70, 4, 264, 20
    d = pre_case(1, B, n, C, iters)
    a, call = pre_run(d, B, n, C, iters, Guarded())
    first = {k: v.clone() for k, v in a.items()}
    call()
    torch.cuda.synchronize()
    b, _ = pre_run(d, B, n, C, iters, Guarded(), in_place=True)
    for k in first:
        assert torch.equal(first[k], a[k]), k  # the same bits again
        assert torch.equal(first[k], b[k]), k


def test_pre_backward_accumulates():
    B, n, C, iters = 70, 2, 72, 5
    K, N = n * C, n * n + 2 * n
    d = pre_case(9, B, n, C, iters)
    plain, _ = pre_run(d, B, n, C, iters, Guarded())
    start = dict(dphi=normal(1, N, K, dtype=F32), dbias=normal(2, N, dtype=F32), dalpha=normal(3, 3, dtype=F32))
    out, _ = pre_run(d, B, n, C, iters, Guarded(), accumulate=1, start=start)
    assert torch.equal(out["dX"], plain["dX"])
    for k, v in start.items():
        assert torch.equal(out[k].cpu(), (v + plain[k].cpu())), k


def test_a_token_without_a_norm_leaves_the_others_alone():
    """r = 0 (its X is zero): its own dX is not finite, every other token's is what it was."""
    B, n, C, iters = 40, 4, 136, 20
    d = pre_case(21, B, n, C, iters)
    clean, _ = pre_run(d, B, n, C, iters, Guarded())
    d["q"][17], d["s"][17], d["Y"][17], d["r"][17] = 0, 10, 0, 0
    out, _ = pre_run(d, B, n, C, iters, Guarded())
    rest = [b for b in range(B) if b != 17]
    assert torch.equal(out["dX"][rest], clean["dX"][rest])
    assert not bool(torch.isfinite(out["dX"][17]).all())


@pytest.mark.parametrize("call", ["dX", "phi", "bias", "alpha", "F"])
def test_gradients_match_differences(call):
    """A whole layer: forward on the GPU, X kept in 8 bits (chosen so that it is kept exactly), both
    backward calls; against central differences of the 64-bit layer along a random direction."""
    B, n, C, iters = 24, 4, 72, 10
    N, K = n * n + 2 * n, n * C
    q, s = pack64(streams(77, B, n, C))
    X = unpack64(q, s)
    v = dict(X=X, F=normal(1, B, C).double(), phi=normal(2, N, K, std=0.05).double(),
             alpha=torch.tensor(ALPHA, dtype=torch.float64), bias=normal(3, N, std=0.5, dtype=F32).double())
    wF, wX = normal(4, B, C, std=1e-2), normal(5, B, n, C, std=1e-2)

    def loss(w):
        F_pre, X_next = layer64(w["X"], w["F"], w["phi"], w["alpha"], w["bias"], iters)
        return float((F_pre * wF.double()).sum() + (X_next * wX.double()).sum())

    dev = {k: t.to(BF).cuda() for k, t in v.items() if k in ("X", "F", "phi")}
    bias = v["bias"].float().cuda()
    o = mhc.alloc_outputs(B, n, C)
    mhc.mhc_gemm_rms_coeffs(dev["X"], dev["phi"], *ALPHA, bias, iters, B, n, C, o["Y"], o["r"], o["H_pre"],
                            o["H_post"], o["H_res"], o["ws"])
    Xq, Xs = mhc.alloc_kept(B, n, C)
    mhc.mhc_post_res_apply_ckpt(dev["X"], dev["F"], o["H_res"], o["H_post"], B, n, C, o["X_next"], Xq, Xs)
    assert torch.equal(unpack64(Xq, Xs), X)
    dF, dhr, dhq = (torch.empty(B, C, dtype=BF, device="cuda"), torch.empty(B, n, n, device="cuda"),
                    torch.empty(B, n, device="cuda"))
    G = wX.cuda()
    mhc.mhc_post_res_apply_backward(G, Xq, Xs, dev["F"], o["H_post"], B, n, C, dF, dhr, dhq)
    got = dict(X=torch.empty(B, n, C, dtype=BF, device="cuda"), phi=torch.empty(N, K, device="cuda"),
               bias=torch.empty(N, device="cuda"), alpha=torch.empty(3, device="cuda"), F=dF)
    mhc.mhc_pre_backward(G, wF.cuda(), Xq, Xs, dev["phi"], *ALPHA, bias, iters, o["Y"], o["r"], o["H_pre"],
                         o["H_post"], o["H_res"], dhr, dhq, 0, B, n, C, got["X"], got["phi"], got["bias"],
                         got["alpha"], mhc.pre_backward_workspace(B, n, C, iters))
    key = {"dX": "X"}.get(call, call)
    d = got[key].double().cpu().view_as(v[key])
    # a random direction; what rounding may do to Σ g·z: bf16 gradients are off by 2^-8 of
    # each term (twice: dY), fp32 ones by the tokens' and channels' chains
    z = normal(6, *v[key].shape, dtype=torch.float64) * (v[key].abs() if key == "X" else 1.0)
    h = 1e-5
    diff = (loss({**v, key: v[key] + h * z}) - loss({**v, key: v[key] - h * z})) / (2 * h)
    mine = float((d * z).sum())
    size = float((d * z).abs().sum())
    rel = 2 * HALF_BF16 if key in ("X", "F") else (C + B + 400) * U32
    assert abs(mine - diff) <= rel * size + 1e-9, (call, mine, diff, size)


# ------------------------------------------------------------- token tables


def make_ids(kind, V, B, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "same":
        return torch.full((B,), V - 1, dtype=torch.int64)
    if kind == "padding":
        return torch.full((B,), -1, dtype=torch.int64)
    u = torch.rand(B, generator=g, dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1.0)) - 1).long().clamp(0, V - 1)
    ids = torch.randperm(V, generator=g)[ids]
    if kind == "ragged":
        bad = torch.rand(B, generator=g) < 0.3
        out = torch.tensor([-1, V, 2 ** 40, -2 ** 40])[torch.randint(0, 4, (B,), generator=g)]
        ids = torch.where(bad, out, ids)
    return ids


EMBED = [("zipf", 1, 1, 1, 8), ("ragged", 100, 15, 4, 72), ("zipf", 100, 16, 4, 72), ("same", 100, 17, 3, 40),
         ("same", 7, 100, 8, 136), ("padding", 50, 40, 2, 40), ("ragged", 1000, 300, 4, 256),
         ("zipf", 20, 700, 5, 72), ("zipf", 200003, 500, 1, 8), ("ragged", 5000, 2000, 2, 264),
         ("ragged", 400, 33, 6, 1000), ("zipf", 64, 130, 7, 2056), ("ragged", 97, 70001, 1, 256),
         ("zipf", 3000, 8200, 1, 2056), ("same", 3, 8200, 1, 2048)]


@pytest.mark.parametrize("ft", [BF, F32])
@pytest.mark.parametrize("kind,V,B,n,C", EMBED)
def test_embed(kind, V, B, n, C, ft):
    ids, T, scale = make_ids(kind, V, B, V + B), normal(3, V, C, std=0.02, dtype=ft), math.sqrt(C)
    g = Guarded()
    X = g.empty(B, n, C, dtype=BF)
    (mhc.mhc_embed if ft == BF else mhc.mhc_embed_f32)(g.put(T), g.put(ids), scale, V, B, n, C, X)
    torch.cuda.synchronize()
    g.check()
    live = (ids >= 0) & (ids < V)
    ref = torch.where(live[:, None], T[ids.clamp(0, V - 1)].double() * scale, torch.zeros((), dtype=torch.float64))
    ref = ref[:, None, :].expand(B, n, C)
    # scale is rounded to fp32, then the product, then to bf16
    within(X, ref, (HALF_BF16 + 3 * U32) * ref.abs(), "X")


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("kind,V,B,n,C", EMBED)
def test_embed_backward(kind, V, B, n, C, accumulate):
    ids, dX, scale = make_ids(kind, V, B, V + B), normal(4, B, n, C, std=1e-2), math.sqrt(C)
    start = normal(5, V, C, std=1e-2, dtype=F32)
    g = Guarded()
    dT = g.put(start) if accumulate else g.empty(V, C)
    ws = g.empty(mhc.embed_backward_workspace(V, B, n, C).numel(), dtype=torch.uint8)
    dXd, idd = g.put(dX), g.put(ids)
    mhc.mhc_embed_backward(dXd, idd, scale, accumulate, V, B, n, C, dT, ws)
    torch.cuda.synchronize()
    g.check()
    live = ((ids >= 0) & (ids < V)).nonzero()[:, 0]
    ref, terms = torch.zeros(V, C, dtype=torch.float64), torch.zeros(V, C, dtype=torch.float64)
    ref.index_add_(0, ids[live], dX[live].double().sum(1) * scale)
    terms.index_add_(0, ids[live], dX[live].double().abs().sum(1) * scale)
    count = torch.zeros(V, dtype=torch.float64).index_add_(0, ids[live], torch.ones(len(live), dtype=torch.float64))
    tol = (n * count[:, None] + 4) * U32 * terms
    if accumulate:
        ref = ref + start.double()
        tol = tol + U32 * (ref.abs() + tol)
        assert torch.equal(dT.cpu()[count == 0], start[count == 0])
    else:
        again = torch.empty(V, C, device="cuda")
        mhc.mhc_embed_backward(dXd, idd, scale, 0, V, B, n, C, again, ws)
        assert torch.equal(again, dT)  # the same bits: the order is fixed
    within(dT, ref, tol, "dtable")


# ------------------------------------------------------- streams and graphs


def test_on_another_stream_and_in_a_graph():
    B, n, C, iters, V = 40, 4, 136, 20, 50
    d = pre_case(31, B, n, C, iters)
    g = Guarded()
    want, _ = pre_run(d, B, n, C, iters, g)
    ids, dX = make_ids("ragged", V, B, 1).cuda(), d["G"].cuda()
    dT, ws = torch.empty(V, C, device="cuda"), mhc.embed_backward_workspace(V, B, n, C)
    mhc.mhc_embed_backward(dX, ids, 2.0, 0, V, B, n, C, dT, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out, call = pre_run(d, B, n, C, iters, g)
        got = torch.empty_like(dT)
    side.synchronize()
    for k in want:
        assert torch.equal(out[k], want[k]), k

    def both():
        call()
        mhc.mhc_embed_backward(dX, ids, 2.0, 0, V, B, n, C, got, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in out:
        out[k].zero_()
    got.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(out[k], want[k]), k
    assert torch.equal(got, dT)


def test_empty_batches():
    n, C, V = 4, 72, 10
    N, K = n * n + 2 * n, n * C
    e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    ws = e(16, dtype=torch.uint8)
    q, s = mhc.alloc_kept(0, n, C)
    for acc in (0, 1):
        dT, dphi, dbias, dalpha = (torch.ones(*x, device="cuda") for x in ((V, C), (N, K), (N,), (3,)))
        mhc.mhc_embed_backward(e(0, n, C, dtype=BF), e(0, dtype=torch.int64), 1.0, acc, V, 0, n, C, dT, ws)
        mhc.mhc_pre_backward(e(0, n, C, dtype=BF), e(0, C, dtype=BF), q, s, e(N, K, dtype=BF), *ALPHA, e(N), 20,
                             e(0, N), e(0), e(0, n), e(0, n), e(0, n, n), e(0, n, n), e(0, n), acc, 0, n, C,
                             e(0, n, C, dtype=BF), dphi, dbias, dalpha, ws)
        for t in (dT, dphi, dbias, dalpha):
            assert bool((t == acc).all())
    mhc.mhc_embed(e(V, C, dtype=BF), e(0, dtype=torch.int64), 1.0, V, 0, n, C, e(0, n, C, dtype=BF))
    mhc.mhc_ckpt_pack(e(0, n, C, dtype=BF), 0, n, C, q, s)


# ---------------------------------------------------------- large and whole


def test_offsets_past_32_bits():
    """More than 2^31 values in X: the last tokens get what they get in a batch of 2500 (which sums
    over channels in the same order)."""
    B, n, C, tail, iters = 76001, 4, 7168, 65, 3
    N, K = n * n + 2 * n, n * C
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s, dtype=F32, std=1.0: torch.randn(*s, device="cuda", generator=gen, dtype=dtype).mul_(std)  # noqa: E731
    X, G, F = rnd(B, n, C, dtype=BF), rnd(B, n, C, dtype=BF, std=1e-2), rnd(B, C, dtype=BF)
    phi, bias = rnd(N, K, dtype=BF, std=0.02), rnd(N, std=0.3)
    Y, r = rnd(B, N), rnd(B).abs() + 0.5
    hp, hq, hr = torch.rand(B, n, device="cuda", generator=gen), rnd(B, n).abs(), rnd(B, n, n).abs()
    dhr, dhq = rnd(B, n, n), rnd(B, n)

    def everything(lo):
        b = B - lo
        cut = lambda t: t[lo:].clone() if lo else t  # noqa: E731
        q, s = mhc.alloc_kept(b, n, C)
        nxt = torch.empty(b, n, C, dtype=BF, device="cuda")
        mhc.mhc_post_res_apply_ckpt(cut(X), cut(F), cut(hr), cut(hq), b, n, C, nxt, q, s)
        dF = torch.empty(b, C, dtype=BF, device="cuda")
        g = [torch.empty(b, n, n, device="cuda"), torch.empty(b, n, device="cuda")]
        mhc.mhc_post_res_apply_backward(cut(G), q, s, cut(F), cut(hq), b, n, C, dF, *g)
        dX = torch.empty(b, n, C, dtype=BF, device="cuda")
        mhc.mhc_pre_backward(cut(G), cut(F), q, s, phi, *ALPHA, bias, iters, cut(Y), cut(r), cut(hp), cut(hq),
                             cut(hr), cut(dhr), cut(dhq), 0, b, n, C, dX, torch.empty(N, K, device="cuda"),
                             torch.empty(N, device="cuda"), torch.empty(3, device="cuda"),
                             mhc.pre_backward_workspace(b, n, C, iters))
        return [t[b - tail:].clone() for t in (nxt, q, s, dF, *g, dX)]

    for a, b in zip(everything(0), everything(B - 2500)):
        assert torch.equal(a, b)


def test_table_offsets_past_32_bits():
    V, C, B, n = 300007, 7168, 40, 1  # 2.15e9 values
    ids = torch.tensor([V - 1, V - 2, V - 1] + list(range(37)), device="cuda")
    T = torch.empty(V, C, dtype=BF, device="cuda")
    T[-2:] = normal(1, 2, C).cuda()
    T[:37] = normal(2, 37, C).cuda()
    X = torch.empty(B, n, C, dtype=BF, device="cuda")
    mhc.mhc_embed(T, ids, 2.0, V, B, n, C, X)
    assert torch.equal(X[:, 0], T[ids] * 2)
    del T
    dT = torch.empty(V, C, device="cuda")
    mhc.mhc_embed_backward(X, ids, 0.5, 0, V, B, n, C, dT, mhc.embed_backward_workspace(V, B, n, C))
    x = X[:, 0].float() * 0.5
    assert torch.equal(dT[V - 1], x[0] + x[2]) and torch.equal(dT[V - 2], x[1])
    assert torch.equal(dT[:37], x[3:]) and not bool(dT[37:V - 2].any())


def test_the_training_example_learns():
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_mhc

    losses = train_mhc.train(steps=40)
    assert abs(losses[0] - math.log(512)) < 1.0  # a uniform guess, nearly
    assert losses[-1] < 0.5 * losses[0]

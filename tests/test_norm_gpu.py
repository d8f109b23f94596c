"""The norms at the entry of F, and their backward, against their formulas in 64 bits.

Tolerances count roundings (train_util).  A thread adds at most 32 squares, a group 5 + 16 partial
sums more, so a sum over channels is off by at most 64 half steps of the sum of magnitudes.
"""
import pytest
import torch

from gpu_util import cuda_ok
from test_train_gpu import normal, streams
from test_train_order_gpu import same_on_poison
from train_util import HALF_BF16, U32, Guarded, pack64, unpack64, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32, F64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8
CHAIN = 64
# one token to many, each number of streams; C of one chunk, odd ones, each layout of the kernels
MIX = [(1, 1, 8), (1, 4, 7168), (3, 2, 40), (9, 3, 72), (33, 4, 264), (65, 4, 1000), (7, 5, 264), (5, 6, 2056),
       (66, 7, 72), (130, 8, 136), (2, 8, 4104), (3, 4, 16384), (2, 8, 8200), (700, 4, 2048), (5, 1, 16376)]
ADD = [(1, 8), (1, 7168), (3, 40), (77, 1000), (33, 264), (600, 256), (5, 2056), (40, 4096), (3, 8200), (2, 16384),
       (2500, 72)]
EPS = 1e-5


def forward64(H, gain, eps, err):
    """(rstd, Z, their tolerances) from H [B, C] in 64 bits, each value off by err at most."""
    ms = H.square().mean(1) + eps
    d_ms = (CHAIN + 2) * U32 * ms + 2.02 * (H.abs() * err).mean(1)
    rstd = ms ** -0.5
    rel = 0.51 * d_ms / ms + 3 * U32
    Z = H * rstd[:, None] * gain
    tol = Z.abs() * (3 * U32 + rel[:, None]) + 1.01 * err * rstd[:, None] * gain.abs()
    return rstd, rstd * rel, Z, tol


def check_q8(q, s, Z, tol):
    """Codes and scales of values within tol of Z: the scale fits the block's largest value, and every
    code stands for what is nearest."""
    q, s = q.cpu(), s.cpu()
    B, C = Z.shape
    nb = -(-C // 32)
    pad = lambda x: torch.nn.functional.pad(x, (0, nb * 32 - C)).view(B, nb, 32)  # noqa: E731
    lo, hi = pad((Z.abs() - tol).clamp_min(0)).amax(-1), pad(Z.abs() + tol).amax(-1)
    scale = torch.exp2(s.double() - 127)
    assert bool((lo <= 448 * scale).all()), "a scale too small"
    assert bool(((hi > 224 * scale) | (s == 10)).all()), "a scale too large"
    got = unpack64(q[:, None], s[:, None])[:, 0]
    step = scale.repeat_interleave(32, -1)[:, :C]
    bound = torch.maximum(2.0 ** -4 * (Z.abs() + tol), 2.0 ** -10 * step) + tol
    over = ((got - Z).abs() - bound).max()
    assert bool(over <= 0), "a code off by %.3e too much" % float(over)


def outputs(g, B, C, q8, keep):
    H, rstd = (g.empty(B, C, dtype=BF), g.empty(B)) if keep else (None, None)
    Z = (g.empty(B, C, dtype=U8), g.empty(B, -(-C // 32), dtype=U8)) if q8 else (g.empty(B, C, dtype=BF),)
    return H, rstd, Z


def check_outputs(H, rstd, Z, H64, gain, eps, err):
    r, r_tol, z, z_tol = forward64(H64, gain.double(), eps, err)
    if H is not None:
        within(H, H64, HALF_BF16 * H64.abs() + 1.01 * err, "H")
        within(rstd, r, r_tol, "rstd")
    if len(Z) == 2:
        check_q8(*Z, z, z_tol)
    else:
        within(Z[0], z, HALF_BF16 * z.abs() + 1.01 * z_tol, "Z")


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,n,C", MIX)
def test_pre_apply_rmsnorm(B, n, C, q8, keep):
    X, gain = streams(B + n + C, B, n, C), 1 + normal(1, C, std=0.2, dtype=F32)
    h = torch.sigmoid(normal(2, B, n, dtype=F64)).float()
    g = Guarded()
    Xd, hd = g.put(X), g.put(h)
    H, rstd, Z = outputs(g, B, C, q8, keep)
    f = mhc.mhc_pre_apply_rmsnorm_q8 if q8 else mhc.mhc_pre_apply_rmsnorm
    f(Xd, hd, g.put(gain), EPS, B, n, C, H, rstd, *Z)
    torch.cuda.synchronize()
    g.check()
    terms = h.double()[:, :, None] * X.double()
    check_outputs(H, rstd, Z, terms.sum(1), gain, EPS, n * U32 * terms.abs().sum(1))
    if keep:  # step 4a's bits
        F = torch.empty(B, C, dtype=BF, device="cuda")
        mhc.mhc_pre_apply(Xd, hd, B, n, C, F)
        assert torch.equal(F, H)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,n,C", [(33, 4, 264), (3, 8, 8200), (40, 0, 2056)])
def test_either_of_what_the_backward_needs_alone(B, n, C, q8):
    """n = 0: a residual's sum.  What is written does not depend on what else is."""
    g = Guarded()
    X, R = g.put(streams(B + C, B, max(n, 1), C)), g.put(streams(C, B, 1, C)[:, 0])
    gain, h = g.put(1 + normal(1, C, std=0.2, dtype=F32)), g.put(torch.sigmoid(normal(2, B, max(n, 1))).float())

    def run(H, rstd, Z):
        tail = "_q8" if q8 else ""
        if n:
            getattr(mhc, "mhc_pre_apply_rmsnorm" + tail)(X, h, gain, EPS, B, n, C, H, rstd, *Z)
        else:
            getattr(mhc, "mhc_add_rmsnorm" + tail)(X[:, 0], R, gain, EPS, B, C, H, rstd, *Z)

    all_H, all_rstd, all_Z = outputs(g, B, C, q8, True)
    run(all_H, all_rstd, all_Z)
    for only_H in (False, True):
        H, rstd, Z = outputs(g, B, C, q8, True)
        run(H if only_H else None, None if only_H else rstd, Z)
        torch.cuda.synchronize()
        g.check()
        assert all(torch.equal(a, b) for a, b in zip(Z, all_Z))
        assert torch.equal(H, all_H) if only_H else torch.equal(rstd, all_rstd)


@pytest.mark.parametrize("into", ["new", "A", "R", "none", "alone"])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,C", ADD)
def test_add_rmsnorm(B, C, q8, into):
    A, R = streams(B + C, B, 1, C)[:, 0], streams(3 * B + C, B, 1, C)[:, 0]
    gain = 1 + normal(1, C, std=0.2, dtype=F32)
    g = Guarded()
    Ad, Rd = g.put(A), g.put(R)
    H, rstd, Z = outputs(g, B, C, q8, True)
    H = {"new": H, "A": Ad, "R": Rd}.get(into)
    f = mhc.mhc_add_rmsnorm_q8 if q8 else mhc.mhc_add_rmsnorm
    f(Ad, None if into == "alone" else Rd, g.put(gain), EPS, B, C, H, rstd, *Z)
    torch.cuda.synchronize()
    g.check()
    if into != "A":
        assert torch.equal(Ad.cpu(), A)
    if into != "R":
        assert torch.equal(Rd.cpu(), R)
    H64 = A.double() + (R.double() if into != "alone" else 0)
    err = U32 * H64.abs()
    r, r_tol, z, z_tol = forward64(H64, gain.double(), EPS, err)
    within(rstd, r, r_tol, "rstd")
    check_outputs(H, rstd, Z, H64, gain, EPS, err)


def test_8_bits_at_the_borders_of_the_format():
    """Rows of ±1 with eps = 0 have rstd = 1, so Z is ±gain, exactly: the codes of any fp32 value."""
    blocks = []
    for top in (448.0, 448.00003, 1.75, 1.7500001, 1.0, 3.3895e38, 3.4028234e38, 2.0 ** 127, 2.0 ** -126, 2.0 ** -149,
                2.0 ** -109, 448 * 2.0 ** -117, 450 * 2.0 ** -117, 0.0):
        row = torch.zeros(32, dtype=F64)
        row[0], row[1] = top, -top
        row[2:30] = top * torch.linspace(-1, 1, 28, dtype=F64)
        row[30], row[31] = -0.0, top * 2.0 ** -16
        blocks.append(row)
    ties = torch.arange(32, dtype=F64) * 0.5 + 240.0  # halves of e4m3 steps under 448
    blocks += [ties, -ties, ties * 2.0 ** -14, ties * (1 + 2.0 ** -20)]
    gain = torch.cat(blocks).float()
    C = gain.numel()
    sign = torch.where(torch.arange(C) % 3 == 0, -1.0, 1.0)
    q, s = torch.empty(2, C, dtype=U8, device="cuda"), torch.empty(2, C // 32, dtype=U8, device="cuda")
    A = torch.stack([sign, -sign]).to(BF).cuda()
    mhc.mhc_add_rmsnorm_q8(A, None, gain.cuda(), 0.0, 2, C, None, None, q, s)
    for k, want in enumerate((sign * gain, -sign * gain)):
        rq, rs = pack64(want[None, None])
        assert torch.equal(s[k].cpu(), rs[0, 0]), k
        assert torch.equal(q[k].cpu(), rq[0, 0]), k


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_rows_that_are_not_finite_stay_alone(bad):
    B, C = 3, 1000
    A = streams(5, B, 1, C)[:, 0]
    A[1, 40] = bad
    Z, rstd, gain = torch.empty(B, C, dtype=BF, device="cuda"), torch.empty(B, device="cuda"), torch.ones(C, device="cuda")
    mhc.mhc_add_rmsnorm(A.cuda(), None, gain, EPS, B, C, None, rstd, Z)
    q, s = torch.empty(B, C, dtype=U8, device="cuda"), torch.empty(B, 32, dtype=U8, device="cuda")
    mhc.mhc_add_rmsnorm_q8(A.cuda(), None, gain, EPS, B, C, None, None, q, s)
    assert bool(torch.isfinite(Z[[0, 2]].float()).all()) and bool(torch.isnan(Z[1, 40]))
    assert bool((s[[0, 2]] != 255).all()) and int(s[1, 1]) == 255
    if bad != bad:
        assert bool(torch.isnan(Z[1]).all()) and bool((s[1] == 255).all())
    else:
        assert float(rstd[1]) == 0.0


def test_rows_of_zeros():
    """Padding: zeros stay zeros, with and without eps, forward and backward."""
    B, n, C = 5, 4, 264
    X = streams(7, B, n, C)
    X[1] = 0
    X[4] = 0
    h, gain = torch.full((B, n), 0.25), 1 + normal(1, C, std=0.2, dtype=F32)
    for eps in (EPS, 0.0):
        g = Guarded()
        H, rstd, Z = outputs(g, B, C, False, True)
        mhc.mhc_pre_apply_rmsnorm(g.put(X), g.put(h), g.put(gain), eps, B, n, C, H, rstd, *Z)
        assert not bool(Z[0][[1, 4]].any()) and bool(torch.isfinite(Z[0].float()).all())
        assert bool(torch.isfinite(rstd).all()) and (eps > 0 or not bool(rstd[[1, 4]].any()))
        dZ = normal(3, B, C).cuda()
        dZ[[1, 4]] = 0
        dH, dgain = torch.empty(B, C, dtype=BF, device="cuda"), torch.empty(C, device="cuda")
        mhc.mhc_rmsnorm_backward(dZ, H, gain.cuda(), rstd, None, 0, B, C, dH, dgain, mhc.rmsnorm_backward_workspace(B, C))
        assert not bool(dH[[1, 4]].any()) and bool(torch.isfinite(dH.float()).all()) and bool(torch.isfinite(dgain).all())


# ------------------------------------------------------------------ backward

BACK = [(1, 8), (1, 7168), (3, 40), (9, 72), (77, 1000), (300, 264), (1000, 256), (5, 2056), (33, 4096), (3, 8200),
        (2, 16384), (2500, 72), (700, 2048), (9000, 8)]


def back_case(seed, B, C):
    H = streams(seed, B, 1, C)[:, 0]
    rstd = (H.double().square().mean(1) + EPS).rsqrt().float()
    return dict(H=H, rstd=rstd, dZ=normal(seed + 1, B, C, std=1e-2), skip=normal(seed + 2, B, C, std=1e-2),
                gain=1 + normal(seed + 3, C, std=0.2, dtype=F32))


def back64(d, skip):
    """(dH, dgain) and what they may be off by, without the last rounding of dH."""
    H, dZ, gain, rstd = (d[k].double() for k in ("H", "dZ", "gain", "rstd"))
    r = rstd[:, None]
    t = gain * dZ
    back = r.square() * (t * H).mean(1, keepdim=True)
    extra = d["skip"].double() if skip else torch.zeros_like(H)
    dH = r * (t - H * back) + extra
    tol = 5 * U32 * (r * (t.abs() + (H * back).abs()) + extra.abs())
    tol = tol + 1.01 * r * H.abs() * r.square() * CHAIN * U32 * (t * H).abs().mean(1, keepdim=True)
    each = dZ * H * r
    return dH, tol, each.sum(0), (H.shape[0] + 24) * U32 * each.abs().sum(0)


@pytest.mark.parametrize("skip,into", [(False, "new"), (False, "dZ"), (True, "new"), (True, "dZ"), (True, "skip")])
@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("B,C", BACK)
def test_rmsnorm_backward(B, C, skip, accumulate, into):
    d = back_case(B + C, B, C)
    start = normal(9, C, std=1e-2, dtype=F32)
    g = Guarded()
    dev = {k: g.put(v) for k, v in d.items()}
    dgain = g.put(start) if accumulate else g.empty(C)
    dH = {"new": None, "dZ": dev["dZ"], "skip": dev["skip"]}[into]
    dH = g.empty(B, C, dtype=BF) if dH is None else dH
    ws = g.empty(mhc.rmsnorm_backward_workspace(B, C).numel(), dtype=U8)
    mhc.mhc_rmsnorm_backward(dev["dZ"], dev["H"], dev["gain"], dev["rstd"], dev["skip"] if skip else None, accumulate,
                             B, C, dH, dgain, ws)
    torch.cuda.synchronize()
    g.check()
    want, tol, wg, wg_tol = back64(d, skip)
    within(dH, want, HALF_BF16 * want.abs() + 1.01 * tol, "dH")
    if accumulate:
        wg = wg + start.double()
        wg_tol = wg_tol + U32 * (wg.abs() + wg_tol)
    within(dgain, wg, wg_tol, "dgain")


@pytest.mark.parametrize("B,C", [(7, 264), (3, 2056)])
def test_backward_against_differences(B, C):
    """Σ w·Z along a direction of H and of the gain: differences of the forward's formula in 64 bits."""
    d = back_case(17, B, C)
    dev = {k: v.cuda() for k, v in d.items()}
    dH, dgain = torch.empty(B, C, dtype=BF, device="cuda"), torch.empty(C, device="cuda")
    mhc.mhc_rmsnorm_backward(dev["dZ"], dev["H"], dev["gain"], dev["rstd"], None, 0, B, C, dH, dgain,
                             mhc.rmsnorm_backward_workspace(B, C))
    H, gain, w = d["H"].double(), d["gain"].double(), d["dZ"].double()

    def value(h, s):
        return float((w * h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * s).sum())

    want, tol, wg, wg_tol = back64(d, False)
    v = normal(5, B, C, dtype=F64) * H.abs().mean(1, keepdim=True)
    u = normal(6, C, dtype=F64)
    for got, x, t in ((dH, v, HALF_BF16 * want.abs() + 1.01 * tol), (dgain, u, wg_tol)):
        step = 1e-4
        if x is v:
            diff = (value(H + step * v, gain) - value(H - step * v, gain)) / (2 * step)
        else:
            diff = (value(H, gain + step * u) - value(H, gain - step * u)) / (2 * step)
        got = got.double().cpu()
        # rstd came rounded to fp32; the third derivative's term is step² of the sum of magnitudes
        slack = float((t * x.abs()).sum()) + (4 * U32 + step ** 2) * float((got.abs() * x.abs()).sum() + (w * H).abs().sum())
        assert abs(float((got * x).sum()) - diff) <= slack


def test_backward_is_reproducible_and_walks_batches():
    B, C = 5001, 1000
    d = {k: v.cuda() for k, v in back_case(3, B, C).items()}
    ws = mhc.rmsnorm_backward_workspace(B, C)
    outs = []
    for _ in range(3):
        dH, dgain = torch.empty(B, C, dtype=BF, device="cuda"), torch.empty(C, device="cuda")
        mhc.mhc_rmsnorm_backward(d["dZ"], d["H"], d["gain"], d["rstd"], d["skip"], 0, B, C, dH, dgain, ws)
        outs.append((dH, dgain))
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])


def test_empty_batch():
    C = 72
    e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    for acc in (0, 1):
        dgain = torch.ones(C, device="cuda")
        mhc.mhc_rmsnorm_backward(e(0, C), e(0, C), e(C, dtype=F32), e(0, dtype=F32), None, acc, 0, C, e(0, C), dgain,
                                 e(16, dtype=U8))
        assert bool((dgain == acc).all())
    mhc.mhc_add_rmsnorm(e(0, C), e(0, C), e(C, dtype=F32), EPS, 0, C, None, None, e(0, C))


def test_a_workspace_that_is_too_small_is_refused():
    B, C = 33, 264
    d = {k: v.cuda() for k, v in back_case(3, B, C).items()}
    dH, dgain = torch.empty(B, C, dtype=BF, device="cuda"), torch.empty(C, device="cuda")
    ws = mhc.rmsnorm_backward_workspace(B, C)
    for w in (ws[:-16], None):
        with pytest.raises(mhc.MhcError):
            mhc.mhc_rmsnorm_backward(d["dZ"], d["H"], d["gain"], d["rstd"], None, 0, B, C, dH, dgain, w)


# ------------------------------------------------------- streams, graphs, order, large


def test_on_another_stream_and_in_a_graph():
    B, n, C = 130, 4, 1000
    X, gain, h = streams(1, B, n, C).cuda(), (1 + normal(1, C, std=0.2, dtype=F32)).cuda(), torch.rand(B, n).cuda()
    dZ, skip = normal(4, B, C).cuda(), normal(5, B, C).cuda()
    ws = mhc.rmsnorm_backward_workspace(B, C)
    e = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731

    def make():
        return [e(B, C, dtype=BF), e(B), e(B, C, dtype=BF), e(B, C, dtype=U8), e(B, 32, dtype=U8), e(B, C, dtype=BF), e(C)]

    def call(o):
        mhc.mhc_pre_apply_rmsnorm(X, h, gain, EPS, B, n, C, o[0], o[1], o[2])
        mhc.mhc_add_rmsnorm_q8(o[2], o[0], gain, EPS, B, C, None, None, o[3], o[4])
        mhc.mhc_rmsnorm_backward(dZ, o[0], gain, o[1], skip, 0, B, C, o[5], o[6], ws)

    want, side_out, graph_out = make(), make(), make()
    call(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(side_out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(graph_out)
    for t in graph_out:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, side_out, graph_out):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("B,n,C", [(4001, 4, 1000), (9000, 2, 72), (1, 4, 7168), (2000, 8, 2056), (130, 1, 16384)])
def test_calls_back_to_back(B, n, C):
    """Each call reads what the call before it wrote, over buffers filled with 0xFF."""
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s, dtype=F32, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).to(dtype)  # noqa: E731
    e = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    X0, h0, gain0, dZ = rnd(B, n, C, dtype=BF), rnd(B, n).abs(), 1 + 0.2 * rnd(C), rnd(B, C, dtype=BF)
    X, q, s = e(B, n, C, dtype=BF), *mhc.alloc_kept(B, n, C)
    mhc.mhc_ckpt_pack(X0, B, n, C, q, s)
    H, rstd, Z, Zq, Zs, Zv = (e(B, C, dtype=BF), e(B), e(B, C, dtype=BF), e(B, C, dtype=U8),
                              e(B, -(-C // 32), dtype=U8), e(B, C, dtype=BF))
    dH, dgain, gain = e(B, C, dtype=BF), e(C), e(C)
    ws = mhc.rmsnorm_backward_workspace(B, C)

    def run():
        mhc.mhc_ckpt_unpack(q, s, B, n, C, X)
        mhc.mhc_pre_apply_rmsnorm(X, h0, gain0, EPS, B, n, C, H, rstd, Z)
        mhc.mhc_rmsnorm_backward(dZ, H, gain0, rstd, Z, 0, B, C, dH, gain, ws)
        mhc.mhc_add_rmsnorm_q8(Z, dH, gain, EPS, B, C, H, rstd, Zq, Zs)
        mhc.mhc_ckpt_unpack(Zq, Zs, B, 1, C, Zv)
        mhc.mhc_rmsnorm_backward(dH, H, gain, rstd, Zv, 0, B, C, dH, dgain, ws)

    same_on_poison(run, [X, H, rstd, Z, Zq, Zs, Zv, dH, gain, dgain, ws], [H, rstd, Z, Zv, dH, gain, dgain])


def test_offsets_past_32_bits():
    B, n, C, tail = 76001, 4, 7168, 65
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s, dtype=F32: torch.randn(*s, device="cuda", generator=g, dtype=dtype)  # noqa: E731
    X, h, gain = rnd(B, n, C, dtype=BF), rnd(B, n), rnd(C)

    def everything(lo):
        b = B - lo
        H, rstd = torch.empty(b, C, dtype=BF, device="cuda"), torch.empty(b, device="cuda")
        q, s = torch.empty(b, C, dtype=U8, device="cuda"), torch.empty(b, C // 32, dtype=U8, device="cuda")
        mhc.mhc_pre_apply_rmsnorm_q8(X[lo:], h[lo:].contiguous(), gain, EPS, b, n, C, H, rstd, q, s)
        return [t[b - tail:].clone() for t in (H, rstd, q, s)]

    for a, b in zip(everything(0), everything(B - 2504)):
        assert torch.equal(a, b)
    del X
    B, C = 300001, 7168
    dZ, H, rstd = rnd(B, C, dtype=BF), rnd(B, C, dtype=BF), rnd(B).abs()
    dH, dgain = torch.empty(B, C, dtype=BF, device="cuda"), torch.empty(C, device="cuda")
    mhc.mhc_rmsnorm_backward(dZ, H, gain, rstd, None, 0, B, C, dH, dgain, mhc.rmsnorm_backward_workspace(B, C))
    d = dict(H=H[-tail:].cpu(), dZ=dZ[-tail:].cpu(), rstd=rstd[-tail:].cpu(), gain=gain.cpu())
    want, tol, _, _ = back64(d, False)
    within(dH[-tail:], want, HALF_BF16 * want.abs() + 1.01 * tol, "dH")

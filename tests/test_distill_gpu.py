"""Distillation on the GPU against its definition in 64 bits (distill_util)."""
import math

import pytest
import torch

from distill_util import distill64
from gpu_util import cuda_ok
from test_train_order_gpu import same_on_poison
from train_util import HALF_BF16, U32, Guarded, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
INF = math.inf


def up8(V):
    return -(-V // 8) * 8


def make(seed, B, V, K, dt, rest, inv_tau=1.0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(B, V, generator=g) * spread
    ids = torch.stack([torch.randperm(V, generator=g)[torch.arange(K) % V] for _ in range(B)])
    t = 9 - 1.5 * torch.log(torch.arange(1, K + 1).float()) + 0.5 * torch.randn(B, K, generator=g)
    z.scatter_(1, ids, t + 0.7 * torch.randn(B, K, generator=g))
    t_lse = None
    if rest:
        top = torch.logsumexp(t * inv_tau, 1)
        t_lse = top - torch.log1p(-(0.01 + 0.4 * torch.rand(B, generator=g)))
    return dict(z=z.to(dt), ids=ids, t=t, t_lse=t_lse, dloss=(0.5 + torch.rand(B, generator=g)) / B)


def call(d, ld, inv_tau, g, grad=True, in_place=False, loss=True):
    """Puts d on the device in rows of ld and runs: (loss, dz [B, ld], what the columns past V held)."""
    B, V = d["z"].shape
    K, dt = d["ids"].shape[1], d["z"].dtype
    z = g.empty(B, ld, dtype=dt)
    z[:, :V] = d["z"].cuda()
    past = z[:, V:].clone()
    args = [g.put(d["ids"]), g.put(d["t"]), g.put(d["t_lse"]) if d["t_lse"] is not None else None]
    out = g.empty(B) if loss else None
    tail = "" if dt == BF else "_f32"
    if not grad:
        getattr(mhc, "mhc_distill_loss" + tail)(z, ld, *args, inv_tau, B, V, K, out)
        return out, None, None
    dz = z if in_place else g.empty(B, ld, dtype=dt)
    getattr(mhc, "mhc_distill_loss_backward" + tail)(z, ld, *args, inv_tau, g.put(d["dloss"]), B, V, K, out, dz)
    torch.cuda.synchronize()
    bits = torch.int16 if dt == BF else torch.int32
    assert torch.equal(dz[:, V:].view(bits), past.view(bits)), "columns past V were written"
    if not in_place:
        assert torch.equal(z[:, V:].view(bits), past.view(bits))
        assert torch.equal(z[:, :V].cpu().view(bits), d["z"].view(bits))
    return out, dz, None


def check(d, out, dz, inv_tau):
    loss, l_tol, want, tol = distill64(d["z"], d["ids"], d["t"], d["t_lse"], inv_tau, d["dloss"])
    if out is not None:
        within(out, loss, l_tol, "loss")
    if dz is not None:
        half = HALF_BF16 if dz.dtype == BF else U32
        within(dz[:, :want.shape[1]], want, 1.01 * tol + half * want.abs(), "dz")


# B, V, K, ld - V rounded up: one value to several blocks a row, odd vocabularies, more entries than threads
SHAPES = [(1, 1, 1, 0), (3, 2, 1, 8), (2, 7, 3, 0), (4, 8, 8, 0), (5, 9, 4, 16), (300, 64, 5, 0), (2, 63, 40, 8),
          (33, 1000, 16, 0), (3, 4097, 33, 0), (1, 32000, 16, 0), (160, 4104, 7, 8), (3, 32000, 600, 0),
          (2, 50001, 32, 0), (1, 131072, 128, 0), (2, 160001, 1, 8), (1, 262144, 1024, 0), (155, 40009, 3, 0)]


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("B,V,K,more", SHAPES)
def test_loss_and_gradient(B, V, K, more, dt, rest):
    inv_tau = 0.5 if V % 2 else 1.0
    d = make(V + K, B, V, K, dt, rest, inv_tau)
    g = Guarded()
    ld = up8(V) + more
    out, dz, _ = call(d, ld, inv_tau, g)
    torch.cuda.synchronize()
    g.check()
    check(d, out, dz, inv_tau)
    alone, _, _ = call(d, ld, inv_tau, g, grad=False)
    torch.cuda.synchronize()
    g.check()
    check(d, alone, None, inv_tau)
    _, here, _ = call(d, ld, inv_tau, g, in_place=True, loss=False)
    g.check()
    assert torch.equal(here[:, :V], dz[:, :V])  # the same bits: the order is fixed


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [1000, 70001])
def test_absent_entries_and_rows(V, dt, rest):
    """Ids out of range, t = -inf, rows without any, whatever those rows' logits hold."""
    B, K = 9, 12
    d = make(5, B, V, K, dt, rest)
    d["ids"][0] = -1
    d["ids"][1] = torch.tensor([V, -1, 2 ** 40, -2 ** 40] * 3)
    d["t"][2] = -INF
    d["ids"][3, ::2] = V
    d["t"][4, 1:] = -INF
    d["ids"][5, 1:] = -5
    d["z"][0, 3], d["z"][1, 5], d["z"][2] = math.nan, INF, -INF
    g = Guarded()
    out, dz, _ = call(d, up8(V), 1.0, g)
    g.check()
    for b in range(3):
        assert float(out[b]) == 0.0 and not bool(dz[b, :V].any())
        d["z"][b] = 0  # the 64-bit form sees plain rows there
    check(d, out, dz, 1.0)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("B,V,K", [(4, 50, 9), (2, 70000, 300), (2, 5, 60)])
def test_an_id_that_comes_more_than_once(B, V, K, dt, rest):
    d = make(6, B, V, K, dt, rest)
    d["ids"][0] = d["ids"][0, torch.arange(K) % 3]  # three ids, over and over
    d["ids"][1, K // 2:] = d["ids"][1, :K - K // 2].clone()
    g = Guarded()
    out, dz, _ = call(d, up8(V), 1.0, g)
    g.check()
    check(d, out, dz, 1.0)
    again, dz2, _ = call(d, up8(V), 1.0, g)
    assert torch.equal(out, again) and torch.equal(dz[:, :V], dz2[:, :V])


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("V,K,of", [(1000, 64, 20), (32000, 1024, 600), (131072, 1001, 3), (262144, 130, 64)])
def test_ids_drawn_with_repetition(V, K, of, rest):
    """As a teacher that samples what it keeps draws them: repeats side by side and far apart, of every part
    of a row; and the same bits each time."""
    B, it = 3, 1.0
    d = make(V + of, B, V, K, F32, rest, it)
    g = torch.Generator().manual_seed(K)
    d["ids"] = torch.randperm(V, generator=g)[:of][torch.randint(0, of, (B, K), generator=g)]
    d["ids"][2, 1::2] = -1
    d["ids"][1, :40] = d["ids"][1, 0]
    if rest:  # a sum that leaves something over
        d["t_lse"] = torch.logsumexp(d["t"] * it, 1) + 0.1
    mem = Guarded()
    out, dz, _ = call(d, up8(V), it, mem)
    check(d, out, dz, it)
    fwd, _, _ = call(d, up8(V), it, mem, grad=False)
    check(d, fwd, None, it)
    for _ in range(3):
        again, dz2, _ = call(d, up8(V), it, mem)
        assert torch.equal(out, again) and torch.equal(dz[:, :V], dz2[:, :V])
        assert torch.equal(call(d, up8(V), it, mem, grad=False)[0], fwd)
    mem.check()


@pytest.mark.parametrize("dt", [BF, F32])
def test_a_masked_vocabulary(dt):
    """-inf in z: no share, no gradient; a kept id there makes the loss infinite."""
    B, V, K = 6, 4100, 5
    for rest in (False, True):
        d = make(7, B, V, K, dt, rest)
        keep = torch.zeros(B, V, dtype=torch.bool).scatter_(1, d["ids"], True)
        mask = torch.rand(B, V, generator=torch.Generator().manual_seed(1)) < 0.5
        mask[1] = True  # nothing but the kept entries
        d["z"] = torch.where(mask & ~keep, torch.tensor(-INF, dtype=dt), d["z"])
        d["z"][2, d["ids"][2, 1]] = -INF
        g = Guarded()
        out, dz, _ = call(d, up8(V), 1.0, g)
        g.check()
        assert float(out[2]) == INF
        assert bool(torch.isfinite(dz[:, :V].float()).all())
        assert not bool(dz[:, :V].cpu()[mask & ~keep].any())
        got = torch.where(torch.isinf(out), torch.zeros_like(out), out)
        loss, l_tol, want, tol = distill64(d["z"], d["ids"], d["t"], d["t_lse"], 1.0, d["dloss"])
        loss[2], l_tol[2] = 0, 0
        within(got, loss, l_tol, "loss")
        within(dz[:, :V], want, 1.01 * tol + (HALF_BF16 if dt == BF else U32) * want.abs(), "dz")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("far", [60.0, 300.0, 2000.0])
def test_kept_logits_far_from_the_rest(far, dt):
    """q_rest far below what 1 - Σ q_k, or a sum relative to the kept logits, could hold; and far above."""
    for sign in (1, -1):
        d = make(8, 3, 2000, 6, dt, True)
        d["z"].scatter_(1, d["ids"], (d["t"] * 0.1 + sign * far).to(dt))
        g = Guarded()
        out, dz, _ = call(d, 2000, 1.0, g)
        g.check()
        check(d, out, dz, 1.0)


def test_probabilities_at_the_borders():
    """A teacher whose kept entries hold all, or (rounded) more than all, of its mass; K = V."""
    for V, K in ((40, 40), (40, 5)):
        d = make(9, 4, V, K, F32, True)
        d["t_lse"] = torch.logsumexp(d["t"].double(), 1).float()
        d["t_lse"][1] -= 1e-6
        d["t_lse"][2] += 1e-7
        g = Guarded()
        out, dz, _ = call(d, up8(V), 1.0, g)
        g.check()
        check(d, out, dz, 1.0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [900, 70000])
def test_rows_that_are_not_finite_stay_alone(V, dt):
    d = make(10, 6, V, 4, dt, False)
    d["z"][1, 17] = math.nan
    d["z"][2, V - 1] = INF
    d["z"][3] = -INF
    d["t"][4, 2] = math.nan
    g = Guarded()
    out, dz, _ = call(d, up8(V), 1.0, g)
    g.check()
    for b in (1, 2, 3):
        assert math.isnan(float(out[b])) and bool(torch.isnan(dz[b, :V]).all()), b
    assert math.isnan(float(out[4]))
    for b in (0, 5):
        r = {k: (v[b:b + 1] if v is not None else None) for k, v in d.items()}
        check(r, out[b:b + 1], dz[b:b + 1], 1.0)
    # a NaN at a kept id
    d = make(10, 1, V, 4, dt, False)
    d["z"][0, d["ids"][0, 1]] = math.nan
    out, dz, _ = call(d, up8(V), 1.0, g)
    assert math.isnan(float(out[0])) and bool(torch.isnan(dz[0, :V]).all())


def test_large_logits_and_temperatures():
    for spread, inv_tau in ((1.5, 0.05), (200.0, 1.0), (1.5, 20.0), (1e30, 1.0)):
        d = make(11, 4, 3001, 8, F32, False, inv_tau, spread)
        g = Guarded()
        out, dz, _ = call(d, 3008, inv_tau, g)
        g.check()
        check(d, out, dz, inv_tau)


@pytest.mark.parametrize("inv_tau", [1e-30, 1e4])
@pytest.mark.parametrize("rest", [False, True])
def test_temperatures_far_out(rest, inv_tau):
    """All alike, and one that takes all."""
    B, V, K = 4, 3001, 8
    d = make(12, B, V, K, F32, rest, inv_tau)
    g = Guarded()
    out, dz, _ = call(d, 3008, inv_tau, g)
    g.check()
    check(d, out, dz, inv_tau)


@pytest.mark.parametrize("dt", [BF, F32])
def test_a_vocabulary_masked_by_the_lowest_value(dt):
    """The type's lowest value in place of -inf: the rest's largest logit may be that."""
    B, V, K = 5, 4100, 5
    low = torch.finfo(dt).min
    for rest in (False, True):
        d = make(17, B, V, K, dt, rest, 0.5)
        keep = torch.zeros(B, V, dtype=torch.bool).scatter_(1, d["ids"], True)
        mask = torch.rand(B, V, generator=torch.Generator().manual_seed(1)) < 0.5
        mask[1:3] = True
        d["z"] = torch.where(mask & ~keep, torch.tensor(low, dtype=dt), d["z"])
        d["z"][3] = low  # every logit
        g = Guarded()
        out, dz, _ = call(d, up8(V), 0.5, g)
        g.check()
        check(d, out, dz, 0.5)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
def test_a_teacher_masked_by_the_lowest_value(dt, rest):
    """Times 1/temperature the lowest value is -inf: where it stands for all entries, they are all alike."""
    B, V, K, it = 3, 900, 40, 4.0
    d = make(31, B, V, K, dt, rest, it)
    d["t"][1, 5:] = d["t"][2, 0] = -2e4  # e^(t·inv_tau) is 0
    low = dict(d, t=d["t"].clone())
    low["t"][1, 5:] = low["t"][2, 0] = torch.finfo(F32).min
    if rest:
        d["t_lse"] = low["t_lse"] = torch.logsumexp(d["t"] * it, 1) + 0.2
    else:
        d["t"][0], low["t"][0] = 0.0, torch.finfo(F32).min
    g = Guarded()
    out, dz, _ = call(low, up8(V), it, g)
    check(d, out, dz, it)
    same, same_dz, _ = call(d, up8(V), it, g)
    assert torch.equal(out, same) and torch.equal(dz[:, :V], same_dz[:, :V])
    fwd, _, _ = call(low, up8(V), it, g, grad=False)
    check(d, fwd, None, it)
    g.check()


def test_one_entry_is_cross_entropy():
    B, V = 37, 513
    d = make(12, B, V, 1, F32, False)
    g = Guarded()
    out, dz, _ = call(d, 520, 1.0, g)
    z = d["z"].double().requires_grad_(True)
    loss = torch.nn.functional.cross_entropy(z, d["ids"][:, 0], reduction="none")
    (want,) = torch.autograd.grad((loss * d["dloss"].double()).sum(), z)
    _, l_tol, _, tol = distill64(d["z"], d["ids"], d["t"], None, 1.0, d["dloss"])
    within(out, loss.detach(), l_tol, "loss")
    within(dz[:, :V], want, 1.01 * tol + U32 * want.abs(), "dz")


@pytest.mark.parametrize("rest", [False, True])
def test_gradient_against_differences_of_the_kernels_loss(rest):
    """Along a direction, the kernel's own loss in fp32: a step of 2^-6 leaves its third derivative."""
    B, V, K = 8, 700, 6
    d = make(13, B, V, K, F32, rest)
    d["dloss"] = torch.ones(B)
    v = torch.randn(B, V, generator=torch.Generator().manual_seed(2))
    h = 2.0 ** -6
    g = Guarded()
    _, dz, _ = call(d, up8(V), 1.0, g)
    up, _, _ = call({**d, "z": d["z"] + h * v}, up8(V), 1.0, g, grad=False)
    dn, _, _ = call({**d, "z": d["z"] - h * v}, up8(V), 1.0, g, grad=False)
    diff = (up.double() - dn.double()).cpu() / (2 * h)
    got = (dz[:, :V].double().cpu() * v.double()).sum(1)
    _, l_tol, _, tol = distill64(d["z"], d["ids"], d["t"], d["t_lse"], 1.0, d["dloss"])
    # |third derivative of log Σ exp along v| <= 6·max|v|³, twice with the rest's; z ± h·v is rounded to fp32
    slack = l_tol * 1.5 / h + h ** 2 * 2 * v.abs().amax(1).double() ** 3 + (tol * v.double().abs()).sum(1)
    slack = slack + 2 * U32 / h * (dz[:, :V].double().cpu().abs() * d["z"].double().abs()).sum(1)
    assert bool(((got - diff).abs() <= slack).all())


def test_on_another_stream_and_in_graphs():
    """Two graphs of the same buffers, replayed in turn."""
    B, V, K = 200, 33000, 17
    d = make(14, B, V, K, BF, True)
    z, ids, t, t_lse, dl = (d[k].cuda() for k in ("z", "ids", "t", "t_lse", "dloss"))
    e = lambda: (torch.zeros(B, device="cuda"), torch.zeros(B, V, dtype=BF, device="cuda"))  # noqa: E731

    def run(o):
        mhc.mhc_distill_loss_backward(z, V, ids, t, t_lse, 1.0, dl, B, V, K, *o)

    want, a, b, c = e(), e(), e(), e()
    run(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(a)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, o in zip(graphs, (b, c)):
        with torch.cuda.graph(graph):
            run(o)
    for k in range(4):
        graphs[k % 2].replay()
    torch.cuda.synchronize()
    for o in (a, b, c):
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


@pytest.mark.parametrize("B,V,K", [(2000, 1000, 3), (300, 32000, 32), (3, 131072, 64), (700, 65536, 600)])
def test_calls_back_to_back(B, V, K):
    """The loss reads logits that the call before wrote, over buffers filled with 0xFF; the gradient overwrites them."""
    g = torch.Generator(device="cuda").manual_seed(V)
    src = torch.randn(B, 1, V, device="cuda", generator=g).to(BF)
    q, s = mhc.alloc_kept(B, 1, V)
    mhc.mhc_ckpt_pack(src, B, 1, V, q, s)
    z, loss, loss2, dz = (torch.zeros(B, 1, V, dtype=BF, device="cuda"), torch.zeros(B, device="cuda"),
                          torch.zeros(B, device="cuda"), torch.zeros(B, V, dtype=BF, device="cuda"))
    ids = torch.randint(0, V, (B, K), device="cuda", generator=g)
    t = torch.randn(B, K, device="cuda", generator=g)
    ones = torch.ones(B, device="cuda")

    def run():
        mhc.mhc_ckpt_unpack(q, s, B, 1, V, z)
        mhc.mhc_distill_loss(z.view(B, V), V, ids, t, None, 1.0, B, V, K, loss)
        mhc.mhc_distill_loss_backward(z.view(B, V), V, ids, t, None, 1.0, ones, B, V, K, loss2, dz)
        mhc.mhc_distill_loss_backward(z.view(B, V), V, ids, t, None, 1.0, loss, B, V, K, None, z.view(B, V))

    same_on_poison(run, [z, loss, loss2, dz], [loss, loss2, dz, z])
    # the two calls may add a row up in another order: each is within its own bound of the value
    mhc.mhc_ckpt_unpack(q, s, B, 1, V, z)
    want, tol, _, _ = distill64(z[:4, 0].cpu(), ids[:4].cpu(), t[:4].cpu(), None, 1.0)
    within(loss[:4], want, tol, "loss")
    within(loss2[:4], want, tol, "loss of the backward")


def test_offsets_past_32_bits():
    B, V, K, tail = 17000, 131072, 8, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.empty(B, V, dtype=BF, device="cuda")
    z[-400:] = torch.randn(400, V, device="cuda", generator=g).to(BF)
    z[:-400] = 0
    ids, t = torch.randint(0, V, (B, K), device="cuda", generator=g), torch.randn(B, K, device="cuda", generator=g)
    dl, loss = torch.rand(B, device="cuda", generator=g), torch.empty(B, device="cuda")
    part, dz_part = torch.empty(400, device="cuda"), torch.empty(400, V, dtype=BF, device="cuda")
    mhc.mhc_distill_loss_backward(z[-400:], V, ids[-400:], t[-400:], None, 1.0, dl[-400:], 400, V, K, part, dz_part)
    mhc.mhc_distill_loss_backward(z, V, ids, t, None, 1.0, dl, B, V, K, loss, z)
    assert torch.equal(loss[-tail:], part[-tail:]) and torch.equal(z[-tail:], dz_part[-tail:])
    # a row of zeros: q = 1/V everywhere
    p = torch.softmax(t[0].double(), 0)
    assert abs(float(loss[0]) - float((p * (torch.log(p) + math.log(V))).sum())) < 1e-4


def test_empty_batch_and_refusals():
    e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    mhc.mhc_distill_loss(e(0, 8, dtype=BF), 8, e(0, 1, dtype=torch.int64), e(0, 1), None, 1.0, 0, 8, 1, e(0))
    z, ids, t, loss = torch.zeros(2, 8, device="cuda"), torch.zeros(2, 1, dtype=torch.int64, device="cuda"), e(2, 1), e(4)
    host = torch.zeros(2, 8).pin_memory()
    st = mhc._lib.mhc_distill_loss_f32(host.data_ptr(), 8, ids.data_ptr(), t.data_ptr(), None, 1.0, 2, 8, 1,
                                       loss.data_ptr(), None)
    assert st == mhc.MHC_ERR_INVALID
    with pytest.raises(mhc.MhcError):
        mhc.mhc_distill_loss_f32(z, 8, ids, t, None, 0.0, 2, 8, 1, loss)

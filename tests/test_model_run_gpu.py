"""The norms and distillation as a model runs them: the norm of the streams into F and at the model's end, the
head's product, the loss with its gradient, and back to the streams.  Each stage is held to its formula in 64
bits on what the stage before it gave; one graph of the whole is replayed."""
import pytest
import torch

from distill_util import distill64
from gpu_util import cuda_ok
from test_norm_gpu import EPS, back64, check_q8, forward64
from test_train_gpu import normal, streams
from train_util import HALF_BF16, U32, Guarded, unpack64, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class End:
    """Streams [B, n, C] to a loss a row and the streams' gradient, through a head of V rows."""

    def __init__(self, B, n, C, V, K, seed=0):
        self.size = B, n, C, V, K, -(-V // 8) * 8
        ld = self.size[-1]
        self.g = g = Guarded()
        self.X = g.put(streams(seed, B, n, C))
        self.even, self.gain = g.put(torch.full((B, n), 1.0 / n)), g.put(1 + normal(seed + 1, C, std=0.2, dtype=F32))
        self.W = g.put(normal(seed + 2, V, C, std=C ** -0.5))
        gen = torch.Generator().manual_seed(seed)
        ids = torch.stack([torch.randperm(V, generator=gen)[:K] for _ in range(B)])
        ids[1] = -1
        ids[2, 1:] = V
        t = normal(seed + 3, B, K, std=2.0, dtype=F32)
        self.ids, self.t = g.put(ids), g.put(t)
        self.t_lse = g.put((torch.logsumexp(t.double() * 0.5, 1) + 0.2).float())
        self.each = g.put(torch.full((B,), 1.0 / B))
        e = g.empty
        self.H, self.Z, self.dH = e(B, C, dtype=BF), e(B, C, dtype=BF), e(B, C, dtype=BF)
        self.rstd, self.loss, self.dgain = e(B), e(B), e(C)
        self.z, self.dz = e(B, ld, dtype=BF), e(B, ld, dtype=BF)
        self.ws = e(max(16, mhc.rmsnorm_backward_workspace(B, C).numel()), dtype=U8)
        self.q, self.s = e(B, C, dtype=U8), e(B, -(-C // 32), dtype=U8)
        self.Zq, self.Zsum = e(B, C, dtype=BF), e(B, C, dtype=BF)
        self.z.zero_()

    def run(self):
        B, n, C, V, K, ld = self.size
        mhc.mhc_pre_apply_rmsnorm(self.X, self.even, self.gain, EPS, B, n, C, self.H, self.rstd, self.Z)
        self.z[:, :V] = self.Z @ self.W.t()
        mhc.mhc_distill_loss_backward(self.z, ld, self.ids, self.t, self.t_lse, 0.5, self.each, B, V, K, self.loss, self.dz)
        self.dZ = self.dz[:, :V] @ self.W
        mhc.mhc_rmsnorm_backward(self.dZ, self.H, self.gain, self.rstd, None, 0, B, C, self.dH, self.dgain, self.ws)
        # an 8-bit projection's input from the same sum, a residual inside F added to it
        mhc.mhc_add_rmsnorm_q8(self.Z, self.H, self.gain, EPS, B, C, self.Zsum, None, self.q, self.s)
        mhc.mhc_ckpt_unpack(self.q, self.s, B, 1, C, self.Zq)

    def outputs(self):
        return [self.H, self.Z, self.rstd, self.z, self.loss, self.dz[:, :self.size[3]], self.dH, self.dgain, self.q, self.s,
                self.Zq, self.Zsum]


@pytest.mark.parametrize("B,n,C,V,K", [(9, 4, 264, 1003, 7), (40, 2, 1000, 33000, 20), (5, 8, 2056, 70001, 130)])
def test_the_models_end(B, n, C, V, K):
    m = End(B, n, C, V, K)
    m.run()
    torch.cuda.synchronize()
    m.g.check()
    assert mhc.mhc_device_status() == mhc.MHC_OK
    cpu = lambda t: t.double().cpu()  # noqa: E731
    terms = cpu(m.X) / n
    err = (n + 1) * U32 * terms.abs().sum(1)
    rstd, r_tol, Z, z_tol = forward64(terms.sum(1), cpu(m.gain), EPS, err)
    within(m.rstd, rstd, r_tol, "rstd")
    within(m.Z, Z, HALF_BF16 * Z.abs() + 1.01 * z_tol, "Z")
    loss, l_tol, dz, tol = distill64(m.z[:, :V].cpu(), m.ids.cpu(), m.t.cpu(), m.t_lse.cpu(), 0.5, m.each.cpu())
    within(m.loss, loss, l_tol, "loss")
    within(m.dz[:, :V], dz, HALF_BF16 * dz.abs() + 1.01 * tol, "dz")
    assert float(m.loss[1]) == 0 and not bool(m.dz[1, :V].any()) and not bool(m.dH[1].any())  # no teacher
    d = dict(H=m.H.cpu(), rstd=m.rstd.cpu(), dZ=m.dZ.cpu(), gain=m.gain.cpu())
    dH, h_tol, dgain, g_tol = back64(d, False)
    within(m.dH, dH, HALF_BF16 * dH.abs() + 1.01 * h_tol, "dH")
    within(m.dgain, dgain, g_tol, "dgain")
    total = cpu(m.Z) + cpu(m.H)
    within(m.Zsum, total, (HALF_BF16 + 2 * U32) * total.abs(), "Z + H")
    _, _, Z2, z2_tol = forward64(total, cpu(m.gain), EPS, U32 * total.abs())
    check_q8(m.q, m.s, Z2, z2_tol)
    assert torch.equal(cpu(m.Zq), unpack64(m.q[:, None], m.s[:, None])[:, 0])


def test_one_graph_of_the_whole():
    B, n, C, V, K = 40, 4, 1000, 33000, 20
    m = End(B, n, C, V, K)
    m.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in m.outputs()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.run()
    for t in m.outputs():
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    m.g.check()
    for a, b in zip(m.outputs(), want):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Two runs at the same time, each with buffers of its own."""
    one, two = End(60, 4, 1000, 33000, 20, 1), End(60, 4, 1000, 33000, 20, 2)
    for m in (one, two):
        m.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in m.outputs()] for m in (one, two)]
    lanes = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for m, lane in zip((one, two), lanes):
            with torch.cuda.stream(lane):
                m.run()
    torch.cuda.synchronize()
    for m, w in zip((one, two), want):
        for a, b in zip(m.outputs(), w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("teacher", [1, 4])
def test_the_training_example_runs_with_a_teacher(teacher):
    import math
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_mhc

    losses = train_mhc.train(steps=3, B=64, C=72, vocab=101, teacher=teacher)
    assert len(losses) == 3 and all(math.isfinite(v) and v > 0 for v in losses)


def test_the_examples_head_gives_the_losss_gradients():
    """Head.step against autograd in 64 bits, along a direction: its products are in bf16, so what comes out
    is off by their roundings: Z, the logits, their gradient, dZ, dX once each, 2^-8 of the magnitudes."""
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_mhc

    B, n, C, V = 16, 4, 72, 101
    gen = torch.Generator(device="cuda").manual_seed(0)
    head = train_mhc.Head(B, n, C, V, gen)
    X = torch.randn(B, n, C, device="cuda", generator=gen).to(BF)
    ids = torch.randint(0, V, (B, 1), device="cuda", generator=gen)
    t = torch.zeros(B, 1, device="cuda")
    loss, dX = head.step(X, ids, t)
    x = X.double().cpu().requires_grad_(True)
    W = head.W.to(BF).double().cpu().requires_grad_(True)
    gain = torch.ones(C, dtype=torch.float64, requires_grad=True)
    h = x.mean(1)
    y = h * (h.square().mean(1, keepdim=True) + train_mhc.EPS).rsqrt() * gain
    z = y @ W.t()
    want = torch.nn.functional.cross_entropy(z, ids[:, 0].cpu())
    gx, gw, gg = torch.autograd.grad(want, [x, W, gain])
    want = float(want.detach())
    # a logit is off by 2^-8·(Σ|y·W| + |z|); q by as much relative to itself; the loss by the largest of them
    slack_z = HALF_BF16 * (y.detach().abs() @ W.detach().abs().t() + z.detach().abs()).amax(1)
    assert abs(float(loss) - want) <= float(2 * slack_z.mean()) + 1e-6
    # |d q| <= 2·slack·q, then its own rounding: summed over the vocabulary against |W|, |y|, with 3 roundings behind
    q = torch.softmax(z.detach(), 1)
    dq = ((2 * slack_z[:, None] + 4 * HALF_BF16) * (q + torch.nn.functional.one_hot(ids[:, 0].cpu(), V))) / B
    rows = (dq @ W.detach().abs()) * (h.detach().square().mean(1, keepdim=True) + train_mhc.EPS).rsqrt()
    tol = (rows + rows.mean(1, keepdim=True) * y.detach().abs() ** 2 + (rows * y.detach().abs()).mean(1, keepdim=True) * y.detach().abs()) / n
    tol = tol[:, None, :] + 3 * HALF_BF16 * gx.abs()
    assert bool(((dX.double().cpu() - gx).abs() <= 1.5 * tol).all())
    tol_w = (dq.t() @ y.detach().abs()) * 1.5 + 2 * HALF_BF16 * gw.abs()
    assert bool(((head.dW.double().cpu() - gw).abs() <= tol_w).all())
    tol_g = ((dq @ W.detach().abs()) * y.detach().abs()).sum(0) * 1.5 + 2 * HALF_BF16 * gg.abs()
    assert bool(((head.dgain.double().cpu() - gg).abs() <= tol_g).all())

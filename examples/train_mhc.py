"""Trains a small language model with mHC residual streams, one token batch a step.

The streams, the mixing, their 8-bit keep and every gradient of theirs are the
library's kernels; the layer function F (a gated projection) and the output head
are plain PyTorch, differentiated by autograd.  The task is synthetic: token b+1
is a fixed permutation of token b, so the loss can go from ln(vocabulary) to zero.

    python examples/train_mhc.py --steps 60
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_rms_sinkhorn_gb300 as mhc  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


class Layer:
    """One mHC layer around F(x) = W2 · (tanh(W1 · x̂)), x̂ = x / rms(x)."""

    def __init__(self, B, n, C, iters, gen):
        N, K = n * n + 2 * n, n * C
        self.B, self.n, self.C, self.iters = B, n, C, iters
        normal = lambda *s, std: torch.randn(*s, device="cuda", generator=gen) * std  # noqa: E731
        # fp32 masters; φ and the weights of F are rounded to bf16 for each step
        self.phi, self.bias = normal(N, K, std=0.02), torch.zeros(N, device="cuda")
        self.bias[2 * n:].view(n, n).fill_diagonal_(2.0)  # start near the identity
        self.alpha = torch.full((3,), 0.1, device="cuda")
        self.W = [normal(C, C, std=C ** -0.5), normal(C, C, std=0.1 * C ** -0.5)]
        self.out = mhc.alloc_outputs(B, n, C)
        self.kept = mhc.alloc_kept(B, n, C)
        self.grads = dict(phi=torch.empty(N, K, device="cuda"), bias=torch.empty(N, device="cuda"),
                          alpha=torch.empty(3, device="cuda"))
        self.dH_res = torch.empty(B, n, n, device="cuda")
        self.dH_post = torch.empty(B, n, device="cuda")
        self.dF_out = torch.empty(B, C, dtype=BF, device="cuda")
        self.ws = mhc.pre_backward_workspace(B, n, C, iters)

    def forward(self, X):
        """X [B, n, C] -> X_next, in place: what the backward needs of X is kept in 8 bits."""
        B, n, C, o = self.B, self.n, self.C, self.out
        self.phi_t, self.a = self.phi.to(BF), self.alpha.tolist()
        mhc.mhc_gemm_rms_coeffs(X, self.phi_t, *self.a, self.bias, self.iters, B, n, C, o["Y"], o["r"],
                                o["H_pre"], o["H_post"], o["H_res"], o["ws"])
        mhc.mhc_pre_apply(X, o["H_pre"], B, n, C, o["F_pre"])
        with torch.enable_grad():
            self.x = o["F_pre"].detach().requires_grad_(True)
            self.w = [w.to(BF).requires_grad_(True) for w in self.W]
            x = self.x.float()
            x = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)).to(BF)
            self.F_out = torch.tanh(x @ self.w[0].t()) @ self.w[1].t()
        mhc.mhc_post_res_apply_ckpt(X, self.F_out.detach(), o["H_res"], o["H_post"], B, n, C, X, *self.kept)
        return X

    def backward(self, dX):
        """dX [B, n, C]: the gradient of X_next, turned into that of X in place."""
        B, n, C, o, g = self.B, self.n, self.C, self.out, self.grads
        mhc.mhc_post_res_apply_backward(dX, *self.kept, self.F_out.detach(), o["H_post"], B, n, C,
                                        self.dF_out, self.dH_res, self.dH_post)
        dF_pre, *self.dW = torch.autograd.grad(self.F_out, [self.x, *self.w], self.dF_out)
        mhc.mhc_pre_backward(dX, dF_pre.contiguous(), *self.kept, self.phi_t, *self.a, self.bias, self.iters,
                             o["Y"], o["r"], o["H_pre"], o["H_post"], o["H_res"], self.dH_res, self.dH_post,
                             0, B, n, C, dX, g["phi"], g["bias"], g["alpha"], self.ws)
        return dX

    def parameters(self):
        g = self.grads
        return [(self.phi, g["phi"]), (self.bias, g["bias"]), (self.alpha, g["alpha"])] + [
            (w, d.float()) for w, d in zip(self.W, self.dW)]


class Adam:
    def __init__(self, lr):
        self.lr, self.t, self.state = lr, 0, {}

    def step(self, pairs):
        self.t += 1
        for p, g in pairs:
            m, v = self.state.setdefault(p.data_ptr(), (torch.zeros_like(p), torch.zeros_like(p)))
            m.lerp_(g, 0.1)
            v.lerp_(g.square(), 0.01)
            p.sub_(self.lr * (m / (1 - 0.9 ** self.t)) / ((v / (1 - 0.99 ** self.t)).sqrt() + 1e-8))


def train(steps=60, B=512, n=4, C=256, layers=2, vocab=512, iters=10, lr=3e-3, seed=0, report=None):
    """The losses of `steps` steps."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    net = [Layer(B, n, C, iters, gen) for _ in range(layers)]
    table = torch.randn(vocab, C, device="cuda", generator=gen) * 0.02
    d_table, ws = torch.empty_like(table), mhc.embed_backward_workspace(vocab, B, n, C)
    head = torch.randn(vocab, C, device="cuda", generator=gen) * C ** -0.5
    follows = torch.randperm(vocab, device="cuda", generator=gen)
    scale, adam, losses = math.sqrt(C), Adam(lr), []
    X = torch.empty(B, n, C, dtype=BF, device="cuda")
    for _ in range(steps):
        ids = torch.randint(0, vocab, (B,), device="cuda", generator=gen)
        mhc.mhc_embed_f32(table, ids, scale, vocab, B, n, C, X)
        for layer in net:
            layer.forward(X)
        with torch.enable_grad():
            x, h = X.detach().requires_grad_(True), head.detach().requires_grad_(True)
            y = x.float().mean(1)
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-5)
            loss = torch.nn.functional.cross_entropy(y @ h.t(), follows[ids])
        dX, d_head = torch.autograd.grad(loss, [x, h])
        for layer in reversed(net):
            layer.backward(dX)
        mhc.mhc_embed_backward(dX, ids, scale, 0, vocab, B, n, C, d_table, ws)
        adam.step([(table, d_table), (head, d_head)] + [p for layer in net for p in layer.parameters()])
        losses.append(loss.item())
        if report:
            report(len(losses), losses[-1])
    if mhc.mhc_device_status() != mhc.MHC_OK:
        raise RuntimeError("a bounded wait ran out on the device")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--batch", type=int, default=512)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args()
    train(a.steps, B=a.batch, layers=a.layers,
          report=lambda k, v: print("step %3d  loss %.4f" % (k, v)) if k == 1 or k % 10 == 0 else None)

"""Refusals of the norms and of distillation, on the host: fake addresses that are never dereferenced,
only where no GPU is visible (as in test_abi.py)."""
import inspect
import math

import pytest
import torch

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")
L = mhc._lib

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device addresses: only where no GPU is visible")

P = [0x10000000 * (k + 1) for k in range(24)]  # 16-byte aligned, far apart
NO_DEVICE = mhc.MHC_ERR_CUDA  # valid host arguments reach the device check


def mix(X=P[0], Hp=P[1], gain=P[2], eps=1e-5, B=4, n=4, C=256, H=P[3], rstd=P[4], Z=P[5]):
    return L.mhc_pre_apply_rmsnorm(X, Hp, gain, eps, B, n, C, H, rstd, Z, None)


def mix_q8(X=P[0], Hp=P[1], gain=P[2], eps=1e-5, B=4, n=4, C=256, H=P[3], rstd=P[4], Zq=P[5], Zs=P[6]):
    return L.mhc_pre_apply_rmsnorm_q8(X, Hp, gain, eps, B, n, C, H, rstd, Zq, Zs, None)


def add(A=P[0], R=P[1], gain=P[2], eps=1e-5, B=4, C=256, H=P[3], rstd=P[4], Z=P[5]):
    return L.mhc_add_rmsnorm(A, R, gain, eps, B, C, H, rstd, Z, None)


def add_q8(A=P[0], R=P[1], gain=P[2], eps=1e-5, B=4, C=256, H=P[3], rstd=P[4], Zq=P[5], Zs=P[6]):
    return L.mhc_add_rmsnorm_q8(A, R, gain, eps, B, C, H, rstd, Zq, Zs, None)


def back(dZ=P[0], H=P[1], gain=P[2], rstd=P[3], skip=P[4], acc=0, B=4, C=256, dH=P[5], dgain=P[6], ws=P[7],
         wsb=(1 << 28) + 1):
    return L.mhc_rmsnorm_backward(dZ, H, gain, rstd, skip, acc, B, C, dH, dgain, ws, wsb, None)


def loss(z=P[0], ld=1000, ids=P[1], t=P[2], t_lse=P[3], it=1.0, B=4, V=1000, K=8, out=P[4], f=None):
    return (f or L.mhc_distill_loss)(z, ld, ids, t, t_lse, it, B, V, K, out, None)


def loss_f32(**kw):
    return loss(f=L.mhc_distill_loss_f32, **kw)


def grad(z=P[0], ld=1000, ids=P[1], t=P[2], t_lse=P[3], it=1.0, dl=P[5], B=4, V=1000, K=8, out=P[4], dz=P[6], f=None):
    return (f or L.mhc_distill_loss_backward)(z, ld, ids, t, t_lse, it, dl, B, V, K, out, dz, None)


def grad_f32(**kw):
    return grad(f=L.mhc_distill_loss_backward_f32, **kw)


NORMS, LOSSES = [mix, mix_q8, add, add_q8, back], [loss, loss_f32, grad, grad_f32]
MAY_BE_NULL = {mix: ["H", "rstd"], mix_q8: ["H", "rstd"], add: ["H", "rstd"], add_q8: ["H", "rstd"], back: ["skip"],
               loss: ["t_lse"], loss_f32: ["t_lse"], grad: ["t_lse", "out"], grad_f32: ["t_lse", "out"]}


@pytest.mark.parametrize("call", NORMS)
def test_norm_shapes(call):
    assert call() == NO_DEVICE
    for C in (0, 12, 16392, 1 << 31):
        assert call(C=C) == mhc.MHC_ERR_UNSUPPORTED, C
    assert call(C=16384) == NO_DEVICE and call(C=8) == NO_DEVICE
    assert call(B=-1) == mhc.MHC_ERR_INVALID
    assert call(B=1 << 31) == mhc.MHC_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [mix, mix_q8])
def test_streams(call):
    for n in (-1, 0, 9):
        assert call(n=n) == mhc.MHC_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [mix, mix_q8, add, add_q8])
def test_eps(call):
    for eps in (math.nan, math.inf, -1e-9):
        assert call(eps=eps) == mhc.MHC_ERR_INVALID
    assert call(eps=0.0) == NO_DEVICE


@pytest.mark.parametrize("call", LOSSES)
def test_loss_rules(call):
    assert call() == NO_DEVICE
    for kw in (dict(B=-1), dict(V=0), dict(K=0), dict(K=-3), dict(ld=992), dict(it=0.0), dict(it=-1.0),
               dict(it=math.nan), dict(it=math.inf), dict(it=2.0 ** 65)):
        assert call(**kw) == mhc.MHC_ERR_INVALID, kw
    for kw in (dict(B=1 << 31), dict(V=(1 << 18) + 8, ld=(1 << 18) + 8), dict(K=1025), dict(ld=1004),
               dict(ld=(1 << 24) + 8)):
        assert call(**kw) == mhc.MHC_ERR_UNSUPPORTED, kw
    assert call(it=2.0 ** 64) == NO_DEVICE
    assert call(V=993) == NO_DEVICE and call(K=1024) == NO_DEVICE  # K may be over V


@pytest.mark.parametrize("call", NORMS + LOSSES)
def test_every_pointer_is_checked(call):
    sig = inspect.signature({loss_f32: loss, grad_f32: grad}.get(call, call))
    names = [k for k, p in sig.parameters.items() if p.default in P and k != "ws"]
    assert names
    for k in names:
        null = NO_DEVICE if k in MAY_BE_NULL[call] else mhc.MHC_ERR_INVALID
        if call in (add, add_q8) and k == "R":
            assert call(R=None) == mhc.MHC_ERR_INVALID  # H is then A
            assert call(R=None, H=None) == NO_DEVICE
        else:
            assert call(**{k: None}) == null, k
        assert call(**{k: sig.parameters[k].default + 8}) == mhc.MHC_ERR_ALIGN, k


def test_overlaps():
    for call in (mix, mix_q8):
        assert call(H=P[0]) == mhc.MHC_ERR_INVALID
        assert call(rstd=P[3]) == mhc.MHC_ERR_INVALID
    for call in (add, add_q8):
        assert call(H=P[0]) == NO_DEVICE and call(H=P[1]) == NO_DEVICE
        assert call(H=P[0] + 16) == mhc.MHC_ERR_INVALID
        assert call(H=P[0], R=P[0]) in (mhc.MHC_ERR_INVALID, NO_DEVICE)
    assert mix(Z=P[0]) == mhc.MHC_ERR_INVALID and add(Z=P[0]) == mhc.MHC_ERR_INVALID
    assert add_q8(Zs=P[5]) == mhc.MHC_ERR_INVALID
    assert back(dH=P[0]) == NO_DEVICE and back(dH=P[4]) == NO_DEVICE
    assert back(dH=P[1]) == mhc.MHC_ERR_INVALID and back(dH=P[0] + 16) == mhc.MHC_ERR_INVALID
    assert back(dgain=P[2]) == mhc.MHC_ERR_INVALID
    for call in (grad, grad_f32):
        assert call(dz=P[0]) == NO_DEVICE
        assert call(dz=P[0] + 16) == mhc.MHC_ERR_INVALID
        assert call(dz=P[2]) == mhc.MHC_ERR_INVALID and call(out=P[5]) == mhc.MHC_ERR_INVALID
    assert loss(out=P[0] + 1600) == mhc.MHC_ERR_INVALID


def test_empty_batches():
    for call in (mix, mix_q8, add, add_q8, loss, loss_f32, grad, grad_f32):
        assert call(B=0) == mhc.MHC_OK
    assert back(B=0, acc=1) == mhc.MHC_OK
    assert back(B=0) == NO_DEVICE  # dgain is set to zero
    assert back(B=0, dgain=None) == mhc.MHC_ERR_INVALID


def test_workspace_sizes():
    f = L.mhc_rmsnorm_backward_workspace_bytes
    assert f(4, 256) == 0  # needs a device
    for B, C in ((0, 256), (-1, 256), (4, 12), (4, 16392)):
        assert f(B, C) == 0


def test_the_binding_checks_types():
    t = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on the device
        mhc.mhc_add_rmsnorm(t, t, t, 1e-5, 4, 256, t, t, t)
    with pytest.raises(TypeError):
        mhc.mhc_pre_apply_rmsnorm(t.float(), None, None, 1e-5, 4, 1, 256, None, None, None)
    with pytest.raises(TypeError):
        mhc.mhc_distill_loss(t.float(), 256, None, None, None, 1.0, 4, 256, 1, None)
    with pytest.raises(TypeError):  # ids are int64
        mhc.mhc_distill_loss_backward(None, 256, torch.zeros(4, 1, dtype=torch.int32), None, None, 1.0, None, 4, 256,
                                      1, None, None)

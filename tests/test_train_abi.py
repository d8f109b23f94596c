"""Refusals of the training calls, on the host: fake addresses that are never dereferenced, only
where no GPU is visible (as in test_abi.py)."""
import math

import pytest
import torch

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")
L = mhc._lib

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device addresses: only where no GPU is visible")

P = [0x10000000 * (k + 1) for k in range(24)]  # 16-byte aligned, far apart
NO_DEVICE = mhc.MHC_ERR_CUDA  # valid host arguments reach the device check


def embed(T=P[0], ids=P[1], scale=1.0, V=100, B=4, n=4, C=256, X=P[2], f=None):
    return (f or L.mhc_embed)(T, ids, scale, V, B, n, C, X, None)


def embed_f32(**kw):
    return embed(f=L.mhc_embed_f32, **kw)


def embed_backward(dX=P[0], ids=P[1], scale=1.0, acc=0, V=100, B=4, n=4, C=256, dT=P[2], ws=P[3],
                   wsb=(1 << 28) + 1):
    return L.mhc_embed_backward(dX, ids, scale, acc, V, B, n, C, dT, ws, wsb, None)


def pack(X=P[0], B=4, n=4, C=256, q=P[1], s=P[2]):
    return L.mhc_ckpt_pack(X, B, n, C, q, s, None)


def unpack(q=P[0], s=P[1], B=4, n=4, C=256, X=P[2]):
    return L.mhc_ckpt_unpack(q, s, B, n, C, X, None)


def keep(X=P[0], F=P[1], hr=P[2], hq=P[3], B=4, n=4, C=256, Xn=P[4], q=P[5], s=P[6], f=None):
    return (f or L.mhc_post_res_apply_ckpt)(X, F, hr, hq, B, n, C, Xn, q, s, None)


def keep_f32(**kw):
    return keep(f=L.mhc_post_res_apply_ckpt_f32, **kw)


def post(G=P[0], q=P[1], s=P[2], F=P[3], hq=P[4], B=4, n=4, C=256, dF=P[5], dhr=P[6], dhq=P[7], f=None):
    return (f or L.mhc_post_res_apply_backward)(G, q, s, F, hq, B, n, C, dF, dhr, dhq, None)


def post_f32(**kw):
    return post(f=L.mhc_post_res_apply_backward_f32, **kw)


def pre(G=P[0], dF=P[1], q=P[2], s=P[3], phi=P[4], bias=P[5], iters=20, Y=P[6], r=P[7], hp=P[8], hq=P[9],
        hr=P[10], dhr=P[11], dhq=P[12], acc=0, B=4, n=4, C=256, dX=P[13], dphi=P[14], dbias=P[15],
        dalpha=P[16], ws=P[17], wsb=(1 << 28) + 1):
    return L.mhc_pre_backward(G, dF, q, s, phi, 0.01, 0.01, 0.01, bias, iters, Y, r, hp, hq, hr, dhr, dhq,
                              acc, B, n, C, dX, dphi, dbias, dalpha, ws, wsb, None)


ALL = [embed, embed_f32, embed_backward, pack, unpack, keep, keep_f32, post, post_f32, pre]


@pytest.mark.parametrize("call", ALL)
def test_shapes(call):
    assert call() == NO_DEVICE
    assert call(n=0) == mhc.MHC_ERR_UNSUPPORTED
    assert call(n=9) == mhc.MHC_ERR_UNSUPPORTED
    assert call(C=0) == mhc.MHC_ERR_UNSUPPORTED
    assert call(C=12) == mhc.MHC_ERR_UNSUPPORTED
    assert call(n=8, C=1 << 28) == mhc.MHC_ERR_UNSUPPORTED
    assert call(B=-1) == mhc.MHC_ERR_INVALID
    assert call(B=1 << 31) == mhc.MHC_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", ALL)
def test_every_pointer_is_checked(call):
    import inspect

    sig = inspect.signature({embed_f32: embed, keep_f32: keep, post_f32: post}.get(call, call))
    names = [k for k, p in sig.parameters.items() if p.default in P and k != "ws"]
    assert names
    for k in names:
        assert call(**{k: None}) == mhc.MHC_ERR_INVALID, k
        assert call(**{k: sig.parameters[k].default + 8}) == mhc.MHC_ERR_ALIGN, k


@pytest.mark.parametrize("call", [embed, embed_f32, embed_backward])
def test_table_rules(call):
    assert call(V=0) == mhc.MHC_ERR_INVALID
    assert call(V=1 << 31) == mhc.MHC_ERR_UNSUPPORTED
    for scale in (math.nan, math.inf, -math.inf):
        assert call(scale=scale) == mhc.MHC_ERR_INVALID


def test_overlaps():
    assert embed(X=P[0] + 1024) == mhc.MHC_ERR_INVALID
    assert embed_backward(dT=P[0]) == mhc.MHC_ERR_INVALID
    assert pack(q=P[0] + 64) == mhc.MHC_ERR_INVALID
    assert pack(s=P[1] + 64) == mhc.MHC_ERR_INVALID  # two outputs
    assert unpack(X=P[0]) == mhc.MHC_ERR_INVALID
    assert keep(Xn=P[0]) == NO_DEVICE  # exactly X
    assert keep(Xn=P[0] + 16) == mhc.MHC_ERR_INVALID
    assert keep(q=P[0]) == mhc.MHC_ERR_INVALID
    assert post(dF=P[3]) == mhc.MHC_ERR_INVALID
    assert post(dF=P[0]) == mhc.MHC_ERR_INVALID
    assert pre(dX=P[0]) == NO_DEVICE  # exactly dX_next
    assert pre(dX=P[0] + 16) == mhc.MHC_ERR_INVALID
    assert pre(dphi=P[4]) == mhc.MHC_ERR_INVALID
    assert pre(dbias=P[16]) == mhc.MHC_ERR_INVALID


def test_other_arguments_and_empty_batches():
    assert pre(iters=-1) == mhc.MHC_ERR_INVALID
    for call in (embed, embed_f32, pack, unpack, keep, keep_f32, post, post_f32):
        assert call(B=0) == mhc.MHC_OK
    # nothing to add; or gradients of weights to set to zero, which needs the device
    assert embed_backward(B=0, acc=1) == mhc.MHC_OK and pre(B=0, acc=1) == mhc.MHC_OK
    assert embed_backward(B=0) == NO_DEVICE and pre(B=0) == NO_DEVICE
    assert embed_backward(B=0, dT=None) == mhc.MHC_ERR_INVALID
    assert pre(B=0, dphi=None) == mhc.MHC_ERR_INVALID


def test_workspace_sizes():
    assert L.mhc_embed_backward_workspace_bytes(100, 4, 9, 256) == 0
    assert L.mhc_embed_backward_workspace_bytes(0, 4, 4, 256) == 0
    assert L.mhc_embed_backward_workspace_bytes(100, 0, 4, 256) == 0
    small, large = (L.mhc_embed_backward_workspace_bytes(100, B, 4, 256) for B in (40, 4000))
    assert 0 < small < large
    # positions past 32 bits of bytes
    assert L.mhc_embed_backward_workspace_bytes(100, 1 << 30, 4, 4096) > 1 << 40
    assert L.mhc_pre_backward_workspace_bytes(4, 4, 256, -1) == 0


def test_the_binding_checks_types():
    t = torch.zeros(4, 4, 256, dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on the device
        mhc.mhc_ckpt_pack(t, 4, 4, 256, t, t)
    with pytest.raises(TypeError):
        mhc.mhc_embed_backward(t.float(), ids, 1.0, 0, 10, 4, 4, 256, t, None)
    with pytest.raises(TypeError):
        mhc.mhc_post_res_apply_ckpt(None, t.float(), None, None, 4, 4, 256, None, None, None)

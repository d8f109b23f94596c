"""64-bit forms of the training operators, written from their formulas, and guarded buffers.

Tolerances count roundings.  u = 2^-24 is half a step of fp32 and 2^-8 half a
step of bf16, relative to the value.  A chain of m fp32 additions is off by at
most m·u·Σ|terms|.  A tensor-core step adds 16 exact products to an fp32 sum
after shifting them to the largest, each dropping at most 2^-23 of it: 17·2^-23
of the absolute sum per step.
"""
import torch

U32 = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
MMA_STEP = 17 * 2.0 ** -23
GUARD = 4096


class Guarded:
    """Device buffers between guard bytes of a known pattern."""

    def __init__(self):
        self.all = []

    def empty(self, *shape, dtype=torch.float32):
        size = torch.empty(0, dtype=dtype).element_size()
        count = 1
        for s in shape:
            count *= s
        nbytes = count * size
        pad = -nbytes % 16
        raw = torch.full((GUARD + nbytes + pad + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((raw, nbytes))
        return raw[GUARD:GUARD + nbytes].view(dtype).view(*shape)

    def put(self, t):
        d = self.empty(*t.shape, dtype=t.dtype)
        d.copy_(t)
        return d

    def check(self):
        for raw, nbytes in self.all:
            assert bool((raw[:GUARD] == 0xA5).all()), "written before a buffer"
            assert bool((raw[GUARD + nbytes:] == 0xA5).all()), "written after a buffer"


def within(got, ref, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), "%s: not finite" % what
    over = (got - ref).abs() - tol
    worst = float(over.max()) if over.numel() else -1.0
    assert worst <= 0, "%s: %d values outside, the worst by %.3e (of %.3e allowed)" % (
        what, int((over > 0).sum()), worst,
        float(torch.as_tensor(tol).expand_as(over).flatten()[over.flatten().argmax()]))


def pack64(X):
    """(codes, scale bytes) of X [B, n, C] from the definition, value by value in 64 bits."""
    B, n, C = X.shape
    nb = -(-C // 32)
    x = torch.zeros(B, n, nb * 32, dtype=torch.float64)
    x[..., :C] = X.double().cpu()
    x = x.view(B, n, nb, 32)
    finite = torch.isfinite(x).all(-1)
    amax = torch.where(finite[..., None], x, torch.zeros_like(x)).abs().amax(-1)
    k = torch.full_like(amax, -117.0)
    for e in range(-117, 120):  # the smallest k with amax <= 448·2^k
        k = torch.where(amax > 448.0 * 2.0 ** e, torch.full_like(k, e + 1.0), k)
    # a magnitude that would round to 2^128 is kept as the largest below it
    top = torch.where(k == 120, 240.0, 448.0)[..., None]
    y = (x / torch.exp2(k)[..., None]).clamp(-top, top)
    mag = y.abs()
    ex = torch.floor(torch.log2(mag.clamp_min(2.0 ** -6)))
    m = torch.round(mag / torch.exp2(ex - 3))  # in steps of the value's binade, to even
    up = m == 16
    ex, m = torch.where(up, ex + 1, ex), torch.where(up, torch.full_like(m, 8.0), m)
    code = torch.where(m >= 8, (ex + 7) * 8 + (m - 8), m)
    code = code + 128 * torch.signbit(x).double()
    code = torch.where(finite[..., None], code, torch.full_like(code, 127.0))
    scale = torch.where(finite, k + 127, torch.full_like(k, 255.0))
    return code.view(B, n, nb * 32)[..., :C].to(torch.uint8), scale.to(torch.uint8)


def unpack64(q, s):
    q = q.cpu().long()
    sign = 1.0 - 2.0 * (q >> 7).double()
    e, m = (q >> 3) & 15, (q & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).double()))
    mag = torch.where((q & 127) == 127, torch.full_like(mag, float("nan")), mag)
    return sign * mag * torch.exp2(s.cpu().double() - 127).repeat_interleave(32, -1)[..., :q.shape[-1]]


def sinkhorn64(H, iters):
    P = torch.exp(H)
    for _ in range(iters):
        P = P / P.sum(-1, keepdim=True)
        P = P / P.sum(-2, keepdim=True)
    return P


def coeffs64(Y, r, alpha, bias, iters, n):
    Ht = torch.cat([alpha[0] * Y[:, :n], alpha[1] * Y[:, n:2 * n], alpha[2] * Y[:, 2 * n:]], 1)
    Ht = Ht / r[:, None] + bias
    return (torch.sigmoid(Ht[:, :n]), 2 * torch.sigmoid(Ht[:, n:2 * n]),
            sinkhorn64(Ht[:, 2 * n:].view(-1, n, n), iters))


def layer64(X, F_out, phi_t, alpha, bias, iters):
    """(F_pre, X_next) of one layer in 64 bits, differentiable in every argument."""
    B, n, C = X.shape
    x = X.reshape(B, n * C)
    Y, r = x @ phi_t.t(), x.square().mean(1).sqrt()
    hp, hq, hr = coeffs64(Y, r, alpha, bias, iters, n)
    return torch.einsum("bi,bic->bc", hp, X), hr @ X + hq[:, :, None] * F_out[:, None, :]

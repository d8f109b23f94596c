"""What stands at the entry of the layer function F and at the model's end, as programs run them: cases,
plain forms and 64-bit values.

  mix_norm      the streams mixed into F's input, F_pre = Σ_i H_pre[i]·X[i], and its RMS norm
                Z = F_pre·rstd·gain, rstd = 1/sqrt(mean F_pre² + eps)
  add_norm      a residual's addition H = A + R inside F, and the norm of H
  norm_grad     the norm's backward: dH = rstd·(t − H·rstd²·mean(t·H)) + dH_skip with t = gain·dZ, and
                dgain = Σ_b dZ·H·rstd
  distill       KL divergence of the student's logits from a teacher of which K logits a row are kept
  distill_grad  the same with the logits' gradient, for a known gradient of each row's loss

Z comes in bf16 or in 8 bits: e4m3 codes with a power-of-two scale for each 32 channels.
The teacher's probabilities are those of its kept logits alone, or, with the logarithm of its sum over the
whole vocabulary, p_k of that sum and the rest in one bucket, held against the student's rest.  An entry
with an id outside the vocabulary is absent; a row without entries has loss 0 and gradient 0.
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # one token of a decoding step, into an 8-bit projection
        {"name": "mix_norm 1 token q8", "op": "mix_norm", "B": 1, "n": 4, "C": 7168, "q8": True, "keep": False},
        # the large prefill batch, into an 8-bit projection
        {"name": "mix_norm 16384 q8", "op": "mix_norm", "B": 16384, "n": 4, "C": 7168, "q8": True, "keep": False},
        # training with eight streams, an odd number of tokens: what the backward reads is kept
        {"name": "mix_norm 8191 n8 keep", "op": "mix_norm", "B": 8191, "n": 8, "C": 4096, "q8": False, "keep": True},
        # an odd number of tokens, a width whose last block of 32 is not full
        {"name": "add_norm 77 odd q8", "op": "add_norm", "B": 77, "C": 1000, "q8": True, "keep": True},
        # between F's sublayers, the large batch
        {"name": "add_norm 16384", "op": "add_norm", "B": 16384, "C": 7168, "q8": False, "keep": True},
        # a short sequence's backward
        {"name": "norm_grad 128", "op": "norm_grad", "B": 128, "C": 7168, "skip": True},
        # the large batch's backward
        {"name": "norm_grad 16384", "op": "norm_grad", "B": 16384, "C": 7168, "skip": True},
        # a few rows of an evaluation
        {"name": "distill 3 rows", "op": "distill", "B": 3, "V": 32000, "ld": 32000, "K": 16, "type": "bf16", "rest": False, "pads": False, "tau": 1.0},
        # an evaluation batch of a large vocabulary, the teacher's rest in a bucket
        {"name": "distill 2048 rest", "op": "distill", "B": 2048, "V": 131072, "ld": 131072, "K": 64, "type": "bf16", "rest": True, "pads": False, "tau": 1.0},
        # fp32 logits of an odd vocabulary in padded rows, some rows without a teacher
        {"name": "distill_grad 500 fp32 odd", "op": "distill_grad", "B": 500, "V": 50001, "ld": 50008, "K": 32, "type": "fp32", "rest": False, "pads": True, "tau": 2.0},
        # a training batch at the vocabulary of 32000, odd number of rows, some without a teacher
        {"name": "distill_grad 4095", "op": "distill_grad", "B": 4095, "V": 32000, "ld": 32000, "K": 32, "type": "bf16", "rest": False, "pads": True, "tau": 1.0},
        # the large batch of a large vocabulary, many logits kept, the rest in a bucket
        {"name": "distill_grad 4096 rest", "op": "distill_grad", "B": 4096, "V": 131072, "ld": 131072, "K": 128, "type": "bf16", "rest": True, "pads": False, "tau": 2.0},
    ]


def _size(rng, lo, hi):
    """A whole number from [lo, hi), spread over its logarithm."""
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))


def draw(rng):
    op = rng.choice(["mix_norm", "add_norm", "norm_grad", "distill", "distill_grad"])
    if op in ("distill", "distill_grad"):
        wide = rng.random() < 0.5  # fp32 logits
        V = _size(rng, 64, 160001)
        B = _size(rng, 1, min(4096, 4096 * 131072 // (V * (2 if wide else 1))) + 1)
        K = _size(rng, 1, min(512, V) + 1)
        ld = -(-V // 8) * 8 + 8 * rng.choice([0, 0, 0, 1, 8])
        return {"op": op, "B": B, "V": V, "ld": ld, "K": K, "type": "fp32" if wide else "bf16",
                "rest": rng.random() < 0.5, "pads": rng.random() < 0.5, "tau": rng.choice([1.0, 1.0, 2.0, 4.0])}
    n = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8]) if op == "mix_norm" else 1
    C = 8 * _size(rng, 1, 2049)
    B = _size(rng, 1, min(16384, 16384 * 4 * 7168 // (n * C)) + 1)
    if op == "norm_grad":
        return {"op": op, "B": B, "C": C, "skip": rng.random() < 0.5}
    case = {"op": op, "B": B, "C": C, "q8": rng.random() < 0.5, "keep": rng.random() < 0.5}
    return {**case, "n": n} if op == "mix_norm" else case


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    bf, f32 = torch.bfloat16, torch.float32

    def normal(*shape, std=1.0, dtype=bf):
        return torch.randn(*shape, device="cuda", generator=g, dtype=dtype).mul_(std)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    def empty(*shape, dtype=f32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = dict(case)
    B, op = s["B"], s["op"]
    if op in ("distill", "distill_grad"):
        V, ld, K = s["V"], s["ld"], s["K"]
        # the teacher's kept ids, one from each of K equal parts of the vocabulary, in any order
        part = V // K
        ids = torch.arange(K, device="cuda") * part + (uniform(B, K) * part).long().clamp_(max=part - 1)
        s["ids"] = ids.gather(1, uniform(B, K).argsort(1))
        # its logits, which fall with their rank; the student has learnt some of them
        rank = torch.arange(1, K + 1, device="cuda", dtype=f32)
        s["t"] = 9.0 - 1.5 * rank.log() + 0.5 * normal(B, K, dtype=f32)
        dt = bf if s["type"] == "bf16" else f32
        s["z"] = normal(B, ld, std=1.5, dtype=dt)
        s["z"].scatter_(1, s["ids"], (s["t"] + normal(B, K, std=0.7, dtype=f32)).to(dt))
        s["inv_tau"] = 1.0 / s["tau"]
        top = torch.logsumexp(s["t"] * s["inv_tau"], 1)
        s["t_lse"] = top - torch.log1p(-(0.01 + 0.3 * uniform(B))) if s["rest"] else None
        if s["pads"]:  # rows without a teacher (a prompt), rows with fewer entries
            keep = (uniform(B, 1) * K * 1.5).long()
            none = uniform(B, 1) < 0.1
            s["ids"] = torch.where((torch.arange(K, device="cuda") < keep.clamp(min=1)) & ~none, s["ids"], -1)
        s["loss"] = empty(B)
        if op == "distill_grad":
            s["dloss"] = (0.5 + uniform(B)) / B
            s["dz"] = empty(B, ld, dtype=dt)
        return s

    C = s["C"]
    s["gain"] = 1.0 + 0.2 * normal(C, dtype=f32)

    def tokens(*shape, std=1.0):  # of very different size, as the residual stream has them
        t = normal(B, *shape, std=std)
        t *= torch.exp(math.log(10.0) * (2.0 * uniform(B, *[1] * len(shape)) - 1.0)).to(bf)
        return t

    if op == "norm_grad":
        s["H"] = tokens(C)
        s["rstd"] = torch.rsqrt(s["H"].float().square().mean(1) + EPS)
        s["dZ"] = normal(B, C, std=1e-2)
        s["dH_skip"] = normal(B, C, std=1e-2) if s["skip"] else None
        s["dH"], s["dgain"] = empty(B, C, dtype=bf), empty(C)
        if own:
            import gemm_rms_sinkhorn_gb300 as mhc

            s["ws"] = mhc.rmsnorm_backward_workspace(B, C)
        return s
    if op == "mix_norm":
        n = s["n"]
        s["X"] = tokens(n, C)
        s["H_pre"] = torch.sigmoid(normal(B, n, dtype=f32))
    else:
        s["A"], s["R"] = normal(B, C), tokens(C)
    s["H"], s["rstd"] = (empty(B, C, dtype=bf), empty(B)) if s["keep"] else (None, None)
    s["Z"] = empty(B, C, dtype=bf)
    if s["q8"]:
        s["Zq"], s["Zs"] = empty(B, C, dtype=torch.uint8), empty(B, -(-C // 32), dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ one pass


def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _rounded8(z):
    """z [B, C] in fp32 as its 8-bit form stands for it."""
    B, C = z.shape
    nb = -(-C // 32)
    x = torch.nn.functional.pad(z, (0, nb * 32 - C)).view(B, nb, 32)
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m · 2^e, 0.5 <= m < 1; 448 = 0.875 · 2^9
    k = torch.where(m > 0.875, e - 8, e - 9).clamp(-117, 120)
    k = torch.where(m == 0, torch.full_like(k, -117), k)[..., None]
    q = (x * _pow2(-k)).to(torch.float8_e4m3fn).float() * _pow2(k)
    return q.view(B, nb * 32)[:, :C].to(torch.bfloat16)


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op in ("distill", "distill_grad"):
        return _plain_distill(s)
    if op == "norm_grad":
        H, dZ, rstd = s["H"].float(), s["dZ"].float(), s["rstd"][:, None]
        t = dZ * s["gain"]
        dH = rstd * (t - H * (rstd.square() * (t * H).mean(1, keepdim=True)))
        if s["skip"]:
            dH = dH + s["dH_skip"].float()
        return {"dH": dH.to(torch.bfloat16), "dgain": (dZ * H * rstd).sum(0)}
    if op == "mix_norm":
        H = (s["H_pre"][:, :, None] * s["X"].float()).sum(1)
    else:
        H = s["A"].float() + s["R"].float()
    rstd = torch.rsqrt(H.square().mean(1) + EPS)
    Z = H * rstd[:, None] * s["gain"]
    out = {"Z": _rounded8(Z) if s["q8"] else Z.to(torch.bfloat16)}
    if s["keep"]:
        out["H"], out["rstd"] = H.to(torch.bfloat16), rstd
    return out


def _log_sum_exp(x, inside):
    x = torch.where(inside, x, torch.full_like(x, -math.inf))
    m = x.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    return (m + torch.log(torch.exp(x - m).sum(1, keepdim=True)))


def _plain_distill(s):
    V, rest = s["V"], s["rest"]
    x = s["z"][:, :V].float() * s["inv_tau"]
    here = (s["ids"] >= 0) & (s["ids"] < V)
    some = here.any(1, keepdim=True)
    ids = s["ids"].clamp(0, V - 1)
    zero = torch.zeros_like(s["t"])
    t = s["t"] * s["inv_tau"]
    log_p = t - (s["t_lse"][:, None] if rest else _log_sum_exp(t, here))
    p = torch.where(here, torch.exp(log_p), zero)
    lse = _log_sum_exp(x, torch.ones_like(x, dtype=torch.bool))
    loss = torch.where(here, p * (log_p - (x.gather(1, ids) - lse)), zero).sum(1)
    factor = p.sum(1, keepdim=True)
    if rest:
        kept = torch.zeros_like(x, dtype=torch.int8).scatter_add_(1, ids, here.to(torch.int8)) > 0
        lse_rest = _log_sum_exp(x, ~kept)
        p_rest = (1.0 - factor).clamp(min=0.0)
        live = (p_rest > 0) & torch.isfinite(lse_rest)
        term = p_rest * (torch.log(p_rest) - (lse_rest - lse))
        loss = loss + torch.where(live & some, term, torch.zeros_like(term))[:, 0]
        p_rest = torch.where(live, p_rest, torch.zeros_like(p_rest))
        factor = factor + p_rest
    if s["op"] == "distill":
        return {"loss": loss}
    dz = torch.exp(x - lse) * factor
    if rest:
        dz = dz - torch.where(kept | ~live, torch.zeros_like(x), p_rest * torch.exp(x - lse_rest))
    dz = dz.scatter_add_(1, ids, -p) * (s["dloss"][:, None] * s["inv_tau"])
    dz = torch.where(some, dz, torch.zeros_like(dz))
    return {"loss": loss, "dz": dz.to(s["z"].dtype)}


def _own(s):
    import gemm_rms_sinkhorn_gb300 as mhc

    op, B = s["op"], s["B"]
    if op in ("distill", "distill_grad"):
        tail = "" if s["type"] == "bf16" else "_f32"
        if op == "distill":
            getattr(mhc, "mhc_distill_loss" + tail)(s["z"], s["ld"], s["ids"], s["t"], s["t_lse"], s["inv_tau"],
                                                    B, s["V"], s["K"], s["loss"])
            return {"loss": s["loss"]}
        getattr(mhc, "mhc_distill_loss_backward" + tail)(s["z"], s["ld"], s["ids"], s["t"], s["t_lse"], s["inv_tau"],
                                                         s["dloss"], B, s["V"], s["K"], s["loss"], s["dz"])
        return {"loss": s["loss"], "dz": s["dz"][:, :s["V"]]}
    C = s["C"]
    if op == "norm_grad":
        mhc.mhc_rmsnorm_backward(s["dZ"], s["H"], s["gain"], s["rstd"], s["dH_skip"], 0, B, C, s["dH"], s["dgain"], s["ws"])
        return {"dH": s["dH"], "dgain": s["dgain"]}
    if op == "mix_norm":
        name, args = "mhc_pre_apply_rmsnorm", (s["X"], s["H_pre"], s["gain"], EPS, B, s["n"], C, s["H"], s["rstd"])
    else:
        name, args = "mhc_add_rmsnorm", (s["A"], s["R"], s["gain"], EPS, B, C, s["H"], s["rstd"])
    if s["q8"]:
        getattr(mhc, name + "_q8")(*args, s["Zq"], s["Zs"])
        mhc.mhc_ckpt_unpack(s["Zq"], s["Zs"], B, 1, C, s["Z"])
    else:
        getattr(mhc, name)(*args, s["Z"])
    out = {"Z": s["Z"]}
    if s["keep"]:
        out["H"], out["rstd"] = s["H"], s["rstd"]
    return out


# ------------------------------------------------------------------ the work


def work(case):
    B, op = case["B"], case["op"]
    if op in ("distill", "distill_grad"):
        size = 2 if case["type"] == "bf16" else 4
        logits, small = B * case["V"] * size, B * (12 * case["K"] + (4 if case["rest"] else 0) + 4)
        if op == "distill":
            return {"bytes": logits + small, "flops": 4 * B * case["V"]}
        return {"bytes": 2 * logits + small + 4 * B, "flops": 7 * B * case["V"]}
    E = B * case["C"]
    if op == "norm_grad":
        return {"bytes": 2 * E * (4 if case["skip"] else 3) + 4 * B + 8 * case["C"], "flops": 10 * E}
    n = case.get("n", 2)
    z = 2 * E + (E + B * -(-case["C"] // 32) if case["q8"] else 0)  # the codes, and the values that they stand for
    kept = 2 * E + 4 * B if case["keep"] else 0
    return {"bytes": 2 * n * E + (4 * B * n if op == "mix_norm" else 0) + 4 * case["C"] + z + kept, "flops": 2 * E * (n + 2)}


# ------------------------------------------------------------------ 64 bits


def _eighth64(Z):
    """Z in 64 bits, rounded to 4 significant bits (fewer below 2^-6) in units of its block's scale."""
    out = torch.empty_like(Z)
    for c in range(0, Z.shape[1], 32):
        x = Z[:, c:c + 32]
        amax = x.abs().amax(1, keepdim=True).clamp_min(2.0 ** -200)
        k = torch.ceil(torch.log2(amax / 448.0))
        k = torch.where(amax > 448.0 * torch.exp2(k), k + 1, k)
        k = torch.where(amax <= 448.0 * torch.exp2(k - 1), k - 1, k).clamp(-117, 120)
        y = x * torch.exp2(-k)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3.0)
        out[:, c:c + 32] = torch.round(y / step) * step * torch.exp2(k)
    return out


def _distill64(s):
    B, V, K = s["B"], s["V"], s["K"]
    loss = torch.zeros(B, device="cuda", dtype=torch.float64)
    dz = torch.zeros(B, V, device="cuda", dtype=torch.float64) if s["op"] == "distill_grad" else None
    step = max(1, (1 << 26) // V)
    for i in range(0, B, step):
        r = slice(i, min(i + step, B))
        ids, z = s["ids"][r], s["z"][r, :V].double()
        q = torch.softmax(z / s["tau"], 1)
        p = torch.zeros(ids.shape[0], V + 1, device="cuda", dtype=torch.float64)  # what is absent: the last column
        at = torch.where((ids >= 0) & (ids < V), ids, V)
        t = torch.where(at < V, s["t"][r].double() / s["tau"], -math.inf)
        some = (at < V).any(1)
        norm = s["t_lse"][r].double() if s["rest"] else torch.logsumexp(torch.where(some[:, None], t, 0.0), 1)
        p.scatter_(1, at, torch.exp(t - norm[:, None]))
        p = p[:, :V]
        kept = torch.zeros(ids.shape[0], V + 1, device="cuda", dtype=torch.bool).scatter_(1, at, True)[:, :V]
        part = torch.where(kept, p * torch.log(p / q), 0.0).sum(1)
        goal = p  # the distribution that the student is held against
        if s["rest"]:
            rest, q_rest = (1.0 - p.sum(1)).clamp(min=0.0), torch.where(kept, 0.0, q).sum(1)
            rest = torch.where(q_rest > 0, rest, 0.0)
            part = part + torch.where(rest > 0, rest * torch.log(rest / q_rest), 0.0)
            share = torch.where(rest > 0, rest / q_rest, 0.0)
            goal = torch.where(kept, p, q * share[:, None])
        loss[r] = torch.where(some, part, 0.0)
        if dz is not None:
            d = (q * goal.sum(1, keepdim=True) - goal) * (s["dloss"][r].double() / s["tau"])[:, None]
            dz[r] = torch.where(some[:, None], d, 0.0)
    return {"loss": loss} if dz is None else {"loss": loss, "dz": dz}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("distill", "distill_grad"):
        return _distill64(s)
    gain = s["gain"].double()
    if s["op"] == "norm_grad":
        H, dZ, rstd = s["H"].double(), s["dZ"].double(), s["rstd"].double()
        back = torch.einsum("bc,bc,c->b", dZ, H, gain) / s["C"] * rstd ** 3
        dH = torch.einsum("bc,c,b->bc", dZ, gain, rstd) - H * back[:, None]
        if s["skip"]:
            dH += s["dH_skip"].double()
        return {"dH": dH, "dgain": torch.einsum("bc,bc,b->c", dZ, H, rstd)}
    if s["op"] == "mix_norm":
        H = torch.zeros(s["B"], s["C"], device="cuda", dtype=torch.float64)
        for i in range(s["n"]):
            H += s["H_pre"][:, i, None].double() * s["X"][:, i].double()
    else:
        H = s["A"].double() + s["R"].double()
    rstd = (H.square().sum(1) / s["C"] + EPS) ** -0.5
    Z = torch.einsum("bc,b,c->bc", H, rstd, gain)
    out = {"Z": _eighth64(Z) if s["q8"] else Z}
    if s["keep"]:
        out["H"], out["rstd"] = H, rstd
    return out

"""The training operators of the mHC layer, as a training program runs them: cases, plain forms and
64-bit values.

  embed       token ids to the n residual streams: X[b][i] = scale · table[ids[b]]
  embed_grad  the table's gradient from the streams' gradient
  keep        the residual update X_next = H_res·X + H_post ⊗ F_out, which also keeps X in 8 bits
              for the backward; and X as it was kept
  post_grad   backward of that update: gradients of F_out, H_res and H_post
  pre_grad    backward of everything before the layer function F (F_pre, the coefficients with their
              Sinkhorn iteration, the projection with its RMS): gradients of X, φ, the bias and the α

X is kept as e4m3 codes with a power-of-two scale for each 32 channels of a stream.
"""
import math

import torch

own = False

ALPHA = (0.01, 0.02, 0.03)  # α_pre, α_post, α_res


def listed():
    return [
        # one token into its streams: the start of a single decoding step
        {"name": "embed 1 token", "op": "embed", "B": 1, "n": 4, "C": 7168, "V": 32000, "table": "bf16", "pads": False},
        # a whole batch of 16384 tokens, ragged (some ids are padding), from an fp32 master table
        {"name": "embed 16384 fp32 table", "op": "embed", "B": 16384, "n": 4, "C": 7168, "V": 32000, "table": "fp32", "pads": True},
        # a short sequence of a small model
        {"name": "embed_grad 64 small", "op": "embed_grad", "B": 64, "n": 4, "C": 256, "V": 1000, "table": "bf16", "pads": True},
        # a training batch: some tokens come a thousand times, most of the vocabulary not at all
        {"name": "embed_grad 16384", "op": "embed_grad", "B": 16384, "n": 4, "C": 4096, "V": 32000, "table": "bf16", "pads": False},
        # an odd number of tokens, a width whose last block of 32 is not full
        {"name": "keep 77 odd", "op": "keep", "B": 77, "n": 4, "C": 1000, "fout": "bf16"},
        # the large batch: n = 4, C = 7168
        {"name": "keep 16384", "op": "keep", "B": 16384, "n": 4, "C": 7168, "fout": "bf16"},
        # one token: latency
        {"name": "post_grad 1 token", "op": "post_grad", "B": 1, "n": 4, "C": 7168, "fout": "bf16"},
        # a width of 4096, the layer's output in fp32
        {"name": "post_grad 4096 fp32", "op": "post_grad", "B": 4096, "n": 4, "C": 4096, "fout": "fp32"},
        # eight streams
        {"name": "post_grad 8192 n8", "op": "post_grad", "B": 8192, "n": 8, "C": 4096, "fout": "bf16"},
        # a short sequence
        {"name": "pre_grad 128", "op": "pre_grad", "B": 128, "n": 4, "C": 7168, "iters": 20},
        # eight streams, an odd number of tokens
        {"name": "pre_grad 8191 n8", "op": "pre_grad", "B": 8191, "n": 8, "C": 4096, "iters": 20},
        # the large batch
        {"name": "pre_grad 16384", "op": "pre_grad", "B": 16384, "n": 4, "C": 7168, "iters": 20},
    ]


def _size(rng, lo, hi):
    """A whole number from [lo, hi), spread over its logarithm; 3072 is left out."""
    x = int(math.exp(rng.uniform(math.log(lo), math.log(hi))))
    return x + 1 if x in (384, 3072) else x


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "keep", "post_grad", "pre_grad"])
    n = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8])
    C = 8 * _size(rng, 8, 897)
    most = 16384 * 4 * 7168 * 32 // (n * C * (n * n + 2 * n + 8))  # as much work as the largest listed case
    B = _size(rng, 1, min(16384, most) + 1)
    case = {"op": op, "B": B, "n": n, "C": C}
    if op in ("embed", "embed_grad"):
        case["V"] = _size(rng, 64, min(131072, (32000 * 4096) // C) + 1)
        case["table"] = rng.choice(["bf16", "fp32"]) if op == "embed" else "bf16"
        case["pads"] = rng.random() < 0.5
    elif op == "pre_grad":
        case["iters"] = rng.choice([0, 1, 3, 5, 10, 20, 20, 20])
    else:
        case["fout"] = rng.choice(["bf16", "fp32"])
    return case


# ------------------------------------------------------------------ 8 bits


def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _pack(X):
    """X [B, n, C] to codes [B, n, C] and the scales' exponents + 127, [B, n, ceil(C / 32)]."""
    B, n, C = X.shape
    nb = -(-C // 32)
    x = torch.nn.functional.pad(X.float(), (0, nb * 32 - C)).view(B, n, nb, 32)
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m · 2^e, 0.5 <= m < 1; 448 = 0.875 · 2^9
    k = torch.where(m > 0.875, e - 8, e - 9).clamp(-117, 120)
    k = torch.where(m == 0, torch.full_like(k, -117), k)
    q = (x * _pow2(-k)[..., None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(B, n, nb * 32)[..., :C].contiguous(), (k + 127).to(torch.uint8)


def _unpack(q, s):
    B, n, C = q.shape
    scale = _pow2(s.to(torch.int32) - 127)
    return q.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(32, -1)[..., :C]


# ------------------------------------------------------------------ inputs


def _sinkhorn(A, iters):
    u = torch.ones_like(A[..., 0])
    v = torch.ones_like(A[:, 0])
    for _ in range(iters):
        u = 1.0 / (A * v[:, None, :]).sum(-1)
        v = 1.0 / (A * u[:, :, None]).sum(-2)
    return u[:, :, None] * A * v[:, None, :]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    bf, f32 = torch.bfloat16, torch.float32

    def normal(*shape, std=1.0, dtype=bf):
        return torch.randn(*shape, device="cuda", generator=g, dtype=dtype).mul_(std)

    def empty(*shape, dtype=f32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = dict(case)
    B, n, C = s["B"], s["n"], s["C"]
    op = s["op"]
    if op in ("embed", "embed_grad"):
        V = s["V"]
        # token frequencies fall as 1/rank; the ranks are spread over the vocabulary
        u = torch.rand(B, device="cuda", generator=g, dtype=torch.float64)
        rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
        ids = torch.randperm(V, device="cuda", generator=g)[rank]
        if s["pads"]:
            ids = torch.where(torch.rand(B, device="cuda", generator=g) < 0.05, torch.full_like(ids, -1), ids)
        s["ids"] = ids
        s["scale"] = math.sqrt(C)
        if op == "embed":
            s["T"] = normal(V, C, std=0.02, dtype=bf if s["table"] == "bf16" else f32)
            s["X"] = empty(B, n, C, dtype=bf)
        else:
            s["dX"] = normal(B, n, C, std=1e-2)
            s["dT"] = empty(V, C)
            if own:
                import gemm_rms_sinkhorn_gb300 as mhc

                s["ws"] = mhc.embed_backward_workspace(V, B, n, C)
        return s

    # tokens of very different size, as the residual stream has them
    X = normal(B, n, C)
    X *= torch.exp(math.log(10.0) * (2.0 * torch.rand(B, 1, 1, device="cuda", generator=g) - 1.0)).to(bf)
    if op in ("keep", "post_grad"):
        s["F_out"] = normal(B, C, dtype=bf if s["fout"] == "bf16" else f32)
        s["H_res"] = _sinkhorn(torch.exp(0.3 * normal(B, n, n, dtype=f32)), 20).contiguous()
        s["H_post"] = 2.0 * torch.sigmoid(0.3 * normal(B, n, dtype=f32))
    if op == "keep":
        s["X"] = X
        s["X_next"], s["X_kept"] = empty(B, n, C, dtype=bf), empty(B, n, C, dtype=bf)
        s["Xq"], s["Xs"] = empty(B, n, C, dtype=torch.uint8), empty(B, n, -(-C // 32), dtype=torch.uint8)
        return s
    s["Xq"], s["Xs"] = _pack(X)
    s["G"] = normal(B, n, C, std=1e-2)
    if op == "post_grad":
        s["dF_out"] = torch.empty_like(s["F_out"])
        s["dH_res"], s["dH_post"] = empty(B, n, n), empty(B, n)
        return s
    K, N = n * C, n * n + 2 * n
    s["phi_t"] = normal(N, K, std=0.02)
    s["bias"] = normal(N, std=0.3, dtype=f32)
    x = X.view(B, K).float()
    s["Y"] = x @ s["phi_t"].float().t()
    s["r"] = x.square().mean(-1).sqrt()
    del x
    alpha = torch.tensor([ALPHA[0]] * n + [ALPHA[1]] * n + [ALPHA[2]] * n * n, device="cuda")
    Ht = alpha * s["Y"] / s["r"][:, None] + s["bias"]
    s["H_pre"] = torch.sigmoid(Ht[:, :n]).contiguous()
    s["H_post"] = 2.0 * torch.sigmoid(Ht[:, n:2 * n])
    s["H_res"] = _sinkhorn(torch.exp(Ht[:, 2 * n:]).view(B, n, n), s["iters"]).contiguous()
    s["dF_pre"] = normal(B, C, std=1e-2)
    s["dH_res"] = normal(B, n, n, std=1e-1, dtype=f32)
    s["dH_post"] = normal(B, n, std=1e-1, dtype=f32)
    s["dX"], s["dphi_t"] = empty(B, n, C, dtype=bf), empty(N, K)
    s["dbias"], s["dalpha"] = empty(N), empty(3)
    if own:
        import gemm_rms_sinkhorn_gb300 as mhc

        s["ws"] = mhc.pre_backward_workspace(B, n, C, s["iters"])
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _own(s)
    op, n = s["op"], s["n"]
    if op == "embed":
        live = (s["ids"] >= 0) & (s["ids"] < s["V"])
        rows = s["T"][s["ids"].clamp(0, s["V"] - 1)].float() * s["scale"]
        rows = torch.where(live[:, None], rows, torch.zeros_like(rows)).to(torch.bfloat16)
        return rows[:, None, :].expand(-1, n, -1).contiguous()
    if op == "embed_grad":
        live = (s["ids"] >= 0) & (s["ids"] < s["V"])
        rows = s["dX"].float().sum(1) * s["scale"]
        rows = torch.where(live[:, None], rows, torch.zeros_like(rows))
        dT = torch.zeros(s["V"], s["C"], device="cuda")
        return dT.index_add_(0, s["ids"].clamp(0, s["V"] - 1), rows)
    if op == "keep":
        x = s["X"].float()
        nxt = torch.bmm(s["H_res"], x) + s["H_post"][:, :, None] * s["F_out"].float()[:, None, :]
        return {"X_next": nxt.to(torch.bfloat16), "X_kept": _unpack(*_pack(s["X"])).to(torch.bfloat16)}
    X = _unpack(s["Xq"], s["Xs"])
    G = s["G"].float()
    if op == "post_grad":
        return {"dF_out": (s["H_post"][:, :, None] * G).sum(1).to(s["F_out"].dtype),
                "dH_res": torch.bmm(G, X.transpose(1, 2)),
                "dH_post": (G * s["F_out"].float()[:, None, :]).sum(-1)}
    return _plain_pre_grad(s, X, G)


def _plain_pre_grad(s, X, G):
    B, n, C, iters = s["B"], s["n"], s["C"], s["iters"]
    K = n * C
    dF, Y, inv_r = s["dF_pre"].float(), s["Y"], 1.0 / s["r"][:, None]
    dH_pre = (X * dF[:, None, :]).sum(-1)
    A = ALPHA[2] * (Y[:, 2 * n:] * inv_r) + s["bias"][2 * n:]
    A = A.view(B, n, n)
    if iters > 0:
        A = A - A.amax(-1, keepdim=True)
    A = torch.exp(A)
    D = s["dH_res"]
    us, vs = [], [torch.ones_like(A[:, 0])]
    for _ in range(iters):
        us.append(1.0 / (A * vs[-1][:, None, :]).sum(-1))
        vs.append(1.0 / (A * us[-1][:, :, None]).sum(-2))
    if iters > 0:
        u, v = us[-1][:, :, None], vs[-1][:, None, :]
        dA = u * v * D
        bu, bv = (A * v * D).sum(-1), (A * u * D).sum(-2)
        for t in range(iters - 1, -1, -1):
            bc = -bv * vs[t + 1].square()
            dA = dA + us[t][:, :, None] * bc[:, None, :]
            br = -(bu + (A * bc[:, None, :]).sum(-1)) * us[t].square()
            dA = dA + br[:, :, None] * vs[t][:, None, :]
            bv, bu = (A * br[:, :, None]).sum(-2), torch.zeros_like(bu)
    else:
        dA = D
    hp, hq = s["H_pre"], s["H_post"]
    dHt = torch.cat([dH_pre * hp * (1.0 - hp), s["dH_post"] * hq * (1.0 - 0.5 * hq), (dA * A).view(B, n * n)], 1)
    dbias = dHt.sum(0)
    each = (dHt * (Y * inv_r)).sum(0)
    dalpha = torch.stack([each[:n].sum(), each[n:2 * n].sum(), each[2 * n:].sum()])
    dY = torch.cat([ALPHA[0] * dHt[:, :n], ALPHA[1] * dHt[:, n:2 * n], ALPHA[2] * dHt[:, 2 * n:]], 1) * inv_r
    sx = -(dY * Y).sum(-1, keepdim=True) * inv_r.square() / K
    dX = torch.bmm(s["H_res"].transpose(1, 2), G)
    dX += hp[:, :, None] * dF[:, None, :]
    dX += (dY @ s["phi_t"].float()).view(B, n, C)
    dX += sx[:, :, None] * X
    return {"dX": dX.to(torch.bfloat16), "dphi_t": dY.t() @ X.view(B, K), "dbias": dbias, "dalpha": dalpha}


def _own(s):
    import gemm_rms_sinkhorn_gb300 as mhc

    op, B, n, C = s["op"], s["B"], s["n"], s["C"]
    if op == "embed":
        f = mhc.mhc_embed if s["table"] == "bf16" else mhc.mhc_embed_f32
        f(s["T"], s["ids"], s["scale"], s["V"], B, n, C, s["X"])
        return s["X"]
    if op == "embed_grad":
        mhc.mhc_embed_backward(s["dX"], s["ids"], s["scale"], 0, s["V"], B, n, C, s["dT"], s["ws"])
        return s["dT"]
    if op == "keep":
        f = mhc.mhc_post_res_apply_ckpt if s["fout"] == "bf16" else mhc.mhc_post_res_apply_ckpt_f32
        f(s["X"], s["F_out"], s["H_res"], s["H_post"], B, n, C, s["X_next"], s["Xq"], s["Xs"])
        mhc.mhc_ckpt_unpack(s["Xq"], s["Xs"], B, n, C, s["X_kept"])
        return {"X_next": s["X_next"], "X_kept": s["X_kept"]}
    if op == "post_grad":
        f = mhc.mhc_post_res_apply_backward if s["fout"] == "bf16" else mhc.mhc_post_res_apply_backward_f32
        f(s["G"], s["Xq"], s["Xs"], s["F_out"], s["H_post"], B, n, C, s["dF_out"], s["dH_res"], s["dH_post"])
        return {"dF_out": s["dF_out"], "dH_res": s["dH_res"], "dH_post": s["dH_post"]}
    mhc.mhc_pre_backward(s["G"], s["dF_pre"], s["Xq"], s["Xs"], s["phi_t"], *ALPHA, s["bias"], s["iters"],
                         s["Y"], s["r"], s["H_pre"], s["H_post"], s["H_res"], s["dH_res"], s["dH_post"], 0,
                         B, n, C, s["dX"], s["dphi_t"], s["dbias"], s["dalpha"], s["ws"])
    return {"dX": s["dX"], "dphi_t": s["dphi_t"], "dbias": s["dbias"], "dalpha": s["dalpha"]}


# ------------------------------------------------------------------ the work


def work(case):
    B, n, C, op = case["B"], case["n"], case["C"], case["op"]
    E = B * n * C
    kept = E + B * n * -(-C // 32)
    if op == "embed":
        return {"bytes": 8 * B + min(B, case["V"]) * C * (2 if case["table"] == "bf16" else 4) + 2 * E, "flops": B * C}
    if op == "embed_grad":
        return {"bytes": 8 * B + 2 * E + 4 * case["V"] * C, "flops": E}
    fo = 2 if case.get("fout") == "bf16" else 4
    if op == "keep":
        return {"bytes": 2 * E + fo * B * C + 4 * B * (n * n + n) + 2 * E + kept + 2 * E, "flops": 2 * E * (n + 2)}
    if op == "post_grad":
        return {"bytes": 2 * E + kept + 2 * fo * B * C + 4 * B * (n * n + 2 * n), "flops": 2 * E * (n + 2)}
    N = n * n + 2 * n
    small = 4 * B * (N + 1 + N + n * n + n) + 4 * N + 4 * (N + 3)
    return {"bytes": 2 * E + 2 * B * C + kept + 2 * N * n * C + 2 * E + 4 * N * n * C + small, "flops": 2 * E * (2 * N + n + 3)}


# ------------------------------------------------------------------ 64 bits


def _kept64(q, s):
    """The values that codes and scales stand for, from the bit fields."""
    q = q.long()
    sign = 1.0 - 2.0 * (q >> 7).double()
    e, m = (q >> 3) & 15, (q & 7).double()
    mag = torch.where(e == 0, m / 8.0 * 2.0 ** -6, (1.0 + m / 8.0) * torch.exp2((e - 7).double()))
    scale = torch.exp2(s.double() - 127.0).repeat_interleave(32, -1)[..., :q.shape[-1]]
    return sign * mag * scale


def _keep64(X):
    """X rounded to 4 significant bits (fewer below 2^-6) in units of its block's scale."""
    B, n, C = X.shape
    out = torch.empty(B, n, C, device=X.device, dtype=torch.float64)
    for c in range(0, C, 32):
        x = X[..., c:c + 32].double()
        amax = x.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -200)
        k = torch.ceil(torch.log2(amax / 448.0))
        k = torch.where(amax > 448.0 * torch.exp2(k), k + 1, k)
        k = torch.where(amax <= 448.0 * torch.exp2(k - 1), k - 1, k).clamp(-117, 120)
        y = x * torch.exp2(-k)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3.0)
        out[..., c:c + 32] = torch.round(y / step) * step * torch.exp2(k)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, B, n, C = s["op"], s["B"], s["n"], s["C"]
    step = max(1, (1 << 26) // (n * C))
    parts = [slice(i, min(i + step, B)) for i in range(0, B, step)]
    dev = {"device": "cuda", "dtype": torch.float64}
    if op == "embed":
        out = torch.zeros(B, n, C, **dev)
        at = ((s["ids"] >= 0) & (s["ids"] < s["V"])).nonzero()[:, 0]
        for i in range(n):
            out[at, i] = s["T"][s["ids"][at]].double() * s["scale"]
        return out
    if op == "embed_grad":
        out = torch.zeros(s["V"], C, **dev)
        at = ((s["ids"] >= 0) & (s["ids"] < s["V"])).nonzero()[:, 0]
        for i in range(n):
            out.index_put_((s["ids"][at],), s["dX"][at, i].double(), accumulate=True)
        return out.mul_(s["scale"])
    if op == "keep":
        nxt = torch.empty(B, n, C, **dev)
        for p in parts:
            x, f = s["X"][p].double(), s["F_out"][p].double()
            for i in range(n):
                nxt[p, i] = (s["H_res"][p, i, :, None].double() * x).sum(1) + s["H_post"][p, i, None].double() * f
        return {"X_next": nxt, "X_kept": torch.cat([_keep64(s["X"][p]) for p in parts])}
    if op == "post_grad":
        out = {"dF_out": torch.empty(B, C, **dev), "dH_res": torch.empty(B, n, n, **dev), "dH_post": torch.empty(B, n, **dev)}
        for p in parts:
            x, g, f = _kept64(s["Xq"][p], s["Xs"][p]), s["G"][p].double(), s["F_out"][p].double()
            out["dF_out"][p] = torch.einsum("bi,bic->bc", s["H_post"][p].double(), g)
            out["dH_res"][p] = torch.einsum("bic,bjc->bij", g, x)
            out["dH_post"][p] = torch.einsum("bic,bc->bi", g, f)
        return out
    # the iteration itself is differentiated; the rest is the chain rule
    K, N = n * C, n * n + 2 * n
    Y, r = s["Y"].double(), s["r"].double()
    yr = Y / r[:, None]
    dHt = torch.empty(B, N, **dev)
    H = (ALPHA[2] * yr[:, 2 * n:] + s["bias"][2 * n:].double()).view(B, n, n).requires_grad_(True)
    P = torch.exp(H)
    for _ in range(s["iters"]):
        P = P / P.sum(2, keepdim=True)
        P = P / P.sum(1, keepdim=True)
    dHt[:, 2 * n:] = torch.autograd.grad(P, H, s["dH_res"].double())[0].reshape(B, n * n)
    hp, hq = s["H_pre"].double(), s["H_post"].double()
    dHt[:, n:2 * n] = s["dH_post"].double() * (hq - hq * hq / 2.0)
    for p in parts:
        dh = torch.einsum("bic,bc->bi", _kept64(s["Xq"][p], s["Xs"][p]), s["dF_pre"][p].double())
        dHt[p, :n] = dh * (hp[p] - hp[p] * hp[p])
    each = (dHt * yr).sum(0)
    alpha = torch.tensor([ALPHA[0]] * n + [ALPHA[1]] * n + [ALPHA[2]] * n * n, **dev)
    dY = alpha * dHt / r[:, None]
    dr = -(dY * yr).sum(1)
    out = {"dX": torch.empty(B, n, C, **dev), "dphi_t": torch.zeros(N, K, **dev), "dbias": dHt.sum(0),
           "dalpha": torch.stack([t.sum() for t in each.split([n, n, n * n])])}
    phi = s["phi_t"].double()
    for p in parts:
        x, g = _kept64(s["Xq"][p], s["Xs"][p]), s["G"][p].double()
        out["dphi_t"] += dY[p].t() @ x.view(-1, K)
        dx = torch.einsum("bij,bic->bjc", s["H_res"][p].double(), g)
        dx += torch.einsum("bj,bc->bjc", hp[p], s["dF_pre"][p].double())
        dx += (dY[p] @ phi).view(-1, n, C)
        out["dX"][p] = dx + x * (dr[p] / (K * r[p]))[:, None, None]
    return out

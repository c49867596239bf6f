"""Timed cases of the gated delta rule and of the head norms with rotation.

The operators, per batch row and step t, with a state H (dk, dv) for each value head:

  g_t    = A[h] softplus(dt_raw[t,h] + dt_bias[h])            log decay (A < 0)
  beta_t = beta_scale sigmoid(beta_raw[t,h])
  H'     = exp(g_t) H_{t-1}                                   (0 where reset[t] is set)
  u_t    = beta_t (v_t - H'^T k_t),   H_t = H' + k_t u_t^T
  out_t  = scale H_t^T q_t

q and k have Hk heads, v has Hv = G Hk heads; value head h reads key head h // G.
"fwd" runs a whole sequence, "bwd" gives its gradients, "step" advances stored
states in place by a window of one or a few tokens.

The norms: n = x r with r = (sum x^2 + eps)^-1/2 ("l2") or (mean x^2 + eps)^-1/2
("rms"), then the weight, then the first rot entries rotated by the position's
angle (halves (i, i + rot/2), or neighbours (2i, 2i + 1)), for every head of q
and k, which are slices of one packed projection. "norm_bwd" gives the gradients
of x and of the weights.

With ``own`` true, ``run`` calls the framework's operators; otherwise it computes
them from elementary torch operations in float32 (the delta rule in chunks of 64
tokens, the only serial part being the state's way from chunk to chunk).
"""
import math

import torch

own = False
CHUNK = 64


def listed():
    return [
        # one request answered token by token: a layer of 12 heads, latency alone
        dict(name="step-1x12", op="step", dtype="bf16", B=1, L=1, Hk=12, Hv=12, dk=128, dv=128),
        # a serving batch of 64 requests, 16 heads: the states come from HBM
        dict(name="step-64x16", op="step", dtype="bf16", B=64, L=1, Hk=8, Hv=16, dk=128, dv=128),
        # a short prompt of odd length
        dict(name="fwd-1x37x16", op="fwd", dtype="bf16", B=1, L=37, Hk=8, Hv=16, dk=128, dv=128,
             packed=False, state=True),
        # float32, odd head sizes, a ragged last chunk
        dict(name="fwd-f32-3x333x3", op="fwd", dtype="f32", B=3, L=333, Hk=1, Hv=3, dk=48, dv=80,
             packed=False, state=True),
        # training / prefill of a layer with 1536 value channels
        dict(name="fwd-8x2048x12", op="fwd", dtype="bf16", B=8, L=2048, Hk=6, Hv=12, dk=128, dv=128,
             packed=False, state=False),
        # rows packed with documents of 64 .. 1024 tokens, 2048 value channels
        dict(name="fwd-packed-2x4096x16", op="fwd", dtype="bf16", B=2, L=4096, Hk=16, Hv=16, dk=128, dv=128,
             packed=True, state=False),
        # one very long sequence on few heads (256 value channels)
        dict(name="fwd-long-1x131072x2", op="fwd", dtype="bf16", B=1, L=131072, Hk=2, Hv=2, dk=128, dv=128,
             packed=False, state=True),
        # the training layer's backward pass
        dict(name="bwd-8x2048x12", op="bwd", dtype="bf16", B=8, L=2048, Hk=6, Hv=12, dk=128, dv=128,
             packed=False, state=False),
        # float32 backward, odd head sizes, documents, initial state and its gradient
        dict(name="bwd-f32-2x250x4", op="bwd", dtype="f32", B=2, L=250, Hk=2, Hv=4, dk=48, dv=80,
             packed=True, state=True),
        # the norms of the serving batch's single tokens
        dict(name="norm-64x1x8", op="norm", dtype="bf16", B=64, L=1, Hq=8, Hk=8, d=128, rot=64, kind="l2",
             pairs="half"),
        # the norms of the training layer, gradient and forward
        dict(name="norm-8x2048x12", op="norm", dtype="bf16", B=8, L=2048, Hq=12, Hk=12, d=128, rot=128, kind="rms",
             pairs="half"),
        dict(name="norm-bwd-8x2048x12", op="norm_bwd", dtype="bf16", B=8, L=2048, Hq=12, Hk=12, d=128, rot=64,
             kind="l2", pairs="next"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "bwd", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        d = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 6, 8, 12])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        most = 8 * 2048 * 24 * 128 // ((Hq + Hk) * d)
        tokens = _spread(rng, 1 if op == "norm" else 64, most if dtype == "bf16" else most // 2)
        B = rng.choice([b for b in (1, 2, 3, 8) if b <= tokens])
        return dict(op=op, dtype=dtype, B=B, L=tokens // B, Hq=Hq, Hk=Hk, d=d, rot=rng.choice([0, d // 2, d]),
                    kind=rng.choice(["l2", "rms"]), pairs=rng.choice(["half", "next"]))
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (96, 64), (48, 80), (33, 50), (192, 128)])
    Hk = rng.choice([1, 2, 4, 6, 8])
    Hv = Hk * rng.choice([1, 1, 2, 3])
    if op == "step":
        B = _spread(rng, 1, 64 * 16 * 128 * 128 // (Hv * dk * dv))
        return dict(op=op, dtype=dtype, B=B, L=rng.choice([1, 1, 1, 2, 5]), Hk=Hk, Hv=Hv, dk=dk, dv=dv)
    most = 8 * 2048 * 12 * 128 * 128 // (Hv * dk * dv) // (1 if dtype == "bf16" else 2)
    B = rng.choice([1, 1, 2, 3, 8])
    L = _spread(rng, 2 if op == "fwd" else 64, min(16384 if op == "fwd" else 4096, most // B))
    return dict(op=op, dtype=dtype, B=B, L=L, Hk=Hk, Hv=Hv, dk=dk, dv=dv, packed=rng.choice([True, False]),
                state=rng.choice([True, False]))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device=dev)

    def unit(x):
        return x / x.square().sum(-1, keepdim=True).sqrt()

    B, L = case["B"], case["L"]
    s = dict(case=dict(case))
    if case["op"].startswith("norm"):
        Hq, Hk, d, rot = case["Hq"], case["Hk"], case["d"], case["rot"]
        # one packed projection (q, k, and the values behind them) as a layer's product leaves it
        packed = normal(B, L, (Hq + 2 * Hk) * d).to(dt)
        s["q"] = packed[..., :Hq * d].view(B, L, Hq, d)
        s["k"] = packed[..., Hq * d:(Hq + Hk) * d].view(B, L, Hk, d)
        s["wq"], s["wk"] = 1.0 + 0.1 * normal(d), 1.0 + 0.1 * normal(d)
        P = L + 4096
        angle = torch.outer(torch.arange(P, device=dev, dtype=torch.float64),
                            10000.0 ** (-torch.arange(rot // 2, device=dev, dtype=torch.float64) / max(1, rot // 2)))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        start = torch.randint(0, 4096, (B, 1), generator=gen, device=dev)
        s["positions"] = (start + torch.arange(L, device=dev)).to(torch.int32).contiguous()
        s["eps"] = 1e-6
        if case["op"] == "norm_bwd":
            s["dq_out"], s["dk_out"] = normal(B, L, Hq, d).to(dt), normal(B, L, Hk, d).to(dt)
        return s
    Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
    lead = (B, L)
    s["q"], s["k"] = unit(normal(*lead, Hk, dk)).to(dt), unit(normal(*lead, Hk, dk)).to(dt)
    s["v"] = normal(*lead, Hv, dv).to(dt)
    s["dt_raw"], s["beta_raw"] = normal(*lead, Hv).to(dt), normal(*lead, Hv).to(dt)
    s["dt_bias"] = torch.log(torch.expm1(torch.exp(uniform(math.log(1e-3), math.log(1e-1), Hv))))
    s["A"] = -uniform(1.0, 16.0, Hv)
    s["scale"] = dk ** -0.5
    s["reset"] = s["h0"] = None
    if case["op"] == "step":
        s["h"] = 0.2 * normal(B, Hv, dk, dv)
        return s
    if case["packed"]:
        t = torch.arange(L, device=dev)
        ends = torch.randint(64, 1025, (B, L // 64 + 1), generator=gen, device=dev).cumsum(1)
        first = (t == 0) & (not case["state"])  # a row that goes on with a state starts inside a document
        s["reset"] = ((t[None, :, None] == ends[:, None, :]).any(-1) | first).to(torch.uint8)
    if case["state"]:
        s["h0"] = 0.2 * normal(B, Hv, dk, dv)
    if case["op"] == "bwd":
        s["dout"] = normal(*lead, Hv, dv).to(dt)
        s["dh_last"] = 0.2 * normal(B, Hv, dk, dv) if case["state"] else None
    return s


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "step":
        return _plain_step(s)
    if case["op"] == "fwd":
        out, h = _plain_fwd(s, s["h0"], CHUNK)[:2]
        return dict(out=out.to(s["v"].dtype), h_last=h)
    if case["op"] == "bwd":
        return _plain_bwd(s)
    if case["op"] == "norm":
        return dict(q=_plain_norm(s, s["q"], s["wq"]), k=_plain_norm(s, s["k"], s["wk"]))
    dq, dwq = _plain_norm_bwd(s, s["q"], s["wq"], s["dq_out"])
    dk, dwk = _plain_norm_bwd(s, s["k"], s["wk"], s["dk_out"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _run_own(s, case):
    import selective_state_space_67_amd as ssm

    if case["op"].startswith("norm"):
        kw = dict(wq=s["wq"], wk=s["wk"], kind=case["kind"], eps=s["eps"])
        if case["rot"]:
            kw.update(cos=s["cos"], sin=s["sin"], positions=s["positions"], interleaved=case["pairs"] == "next")
        if case["op"] == "norm":
            q, k = ssm.ssm_qk_norm_fwd(s["q"], s["k"], out_dtype=s["q"].dtype, **kw)
            return dict(q=q, k=k)
        g = ssm.ssm_qk_norm_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], grad_dtype=s["q"].dtype, **kw)
        return dict(dq=g["dq"], dk=g["dk"], dwq=g["dwq"], dwk=g["dwk"])
    a = (s["q"], s["k"], s["v"], s["dt_raw"], s["A"], s["beta_raw"])
    if case["op"] == "step":
        out = ssm.ssm_delta_update(s["h"], *a, dt_bias=s["dt_bias"], scale=s["scale"], out_dtype=s["v"].dtype)
        return dict(out=out, h=s["h"])
    if case["op"] == "fwd":
        h_last = torch.empty((case["B"], case["Hv"], case["dk"], case["dv"]), device=s["v"].device)
        out = ssm.ssm_delta_fwd(*a, dt_bias=s["dt_bias"], reset=s["reset"], h0=s["h0"], h_last=h_last,
                                scale=s["scale"], out_dtype=s["v"].dtype)
        return dict(out=out, h_last=h_last)
    g = ssm.ssm_delta_bwd(*a, s["dout"], dt_bias=s["dt_bias"], reset=s["reset"], h0=s["h0"], dh_last=s["dh_last"],
                          scale=s["scale"], grad_dtype=s["v"].dtype)
    return {k: g[k] for k in ("dq", "dk", "dv", "d_dt_raw", "dbeta_raw", "dA", "d_dt_bias", "dh0")}


# ---- the plain forms ----

def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _unit_lower_inverse(A):
    """(I + A)^-1 for strictly lower A, by doubling the inverted diagonal blocks."""
    C = A.shape[-1]
    i = torch.arange(C, device=A.device)
    X = torch.eye(C, device=A.device).expand_as(A)
    b = 1
    while b < C:
        pair = (i[:, None] // (2 * b) == i[None, :] // (2 * b)) & (i[:, None] // b != i[None, :] // b)
        X = X - X @ (A * pair) @ X
        b *= 2
    return X


def _chunks(s, C):
    """The inputs in float32 as (B, Hv, chunks, C, ..), padded with tokens that do nothing, and each chunk's matrices."""
    B, L, Hk, dk = s["q"].shape
    Hv = s["v"].shape[2]
    n = -(-L // C)

    def cut(x, group=1):
        x = x.float()
        x = torch.cat([x, x.new_zeros((B, n * C - L) + x.shape[2:])], 1) if n * C > L else x
        x = x.movedim(2, 1)
        x = x.repeat_interleave(group, 1) if group > 1 else x
        return x.reshape((B, Hv, n, C) + x.shape[3:]).contiguous()

    G = Hv // Hk
    raw = s["dt_raw"].float() + s["dt_bias"]
    delta = _softplus(raw)
    c = dict(q=cut(s["q"], G) * s["scale"], k=cut(s["k"], G), v=cut(s["v"]), raw=raw, delta=delta,
             beta=cut(torch.sigmoid(s["beta_raw"].float())))
    if s["reset"] is None:
        seg = torch.zeros((B, 1, n, C), device=raw.device)
        g = cut(delta * s["A"])
    else:
        on = s["reset"].bool()
        g = cut(torch.where(on[..., None], torch.zeros_like(delta), delta * s["A"]))
        on = torch.cat([on, on.new_zeros((B, n * C - L))], 1) if n * C > L else on
        seg = on.float().reshape(B, 1, n, C).cumsum(-1)
    sums = g.cumsum(-1)
    i = torch.arange(C, device=raw.device)
    same = (seg[..., :, None] == seg[..., None, :]) & (i[:, None] >= i[None, :])
    diff = (sums[..., :, None] - sums[..., None, :]).masked_fill(~same, -math.inf)
    c["M"] = torch.exp(diff)
    c["e0"] = torch.exp(sums) * (seg == 0)
    c["eC"] = torch.exp(sums[..., -1:] - sums) * (seg == seg[..., -1:])
    c["aC"] = c["e0"][..., -1]
    c["S"] = c["k"] @ c["k"].transpose(-1, -2)
    low = torch.tril(c["M"], -1)
    c["low"] = low
    c["T"] = _unit_lower_inverse(c["beta"][..., None] * low * c["S"])
    c["QK"] = c["q"] @ c["k"].transpose(-1, -2)
    c["P"] = c["M"] * c["QK"]
    c["kC"] = c["eC"][..., None] * c["k"]
    return c


def _plain_fwd(s, h0, C):
    c = _chunks(s, C)
    B, L, Hv, dv = s["v"].shape
    W = c["T"] @ ((c["beta"] * c["e0"])[..., None] * c["k"])
    U0 = c["T"] @ (c["beta"][..., None] * c["v"])
    H = h0 if h0 is not None else U0.new_zeros((B, Hv, s["k"].shape[3], dv))
    starts, us = [], []
    for j in range(W.shape[2]):
        starts.append(H)
        U = U0[:, :, j] - W[:, :, j] @ H
        us.append(U)
        H = c["aC"][:, :, j, None, None] * H + c["kC"][:, :, j].transpose(-1, -2) @ U
    starts, U = torch.stack(starts, 2), torch.stack(us, 2)
    out = c["e0"][..., None] * (c["q"] @ starts) + c["P"] @ U
    return out.reshape(B, Hv, -1, dv)[:, :, :L].transpose(1, 2).contiguous(), H, c, starts, U


def _plain_step(s):
    B, L, Hk, dk = s["q"].shape
    Hv = s["v"].shape[2]
    alpha = torch.exp(s["A"] * _softplus(s["dt_raw"].float() + s["dt_bias"]))[..., None, None]
    beta = torch.sigmoid(s["beta_raw"].float())[..., None]
    q, k = (s["q"].float() * s["scale"], s["k"].float())
    if Hv > Hk:
        q, k = q.repeat_interleave(Hv // Hk, 2), k.repeat_interleave(Hv // Hk, 2)
    v, H, outs = s["v"].float(), s["h"], []
    for t in range(L):
        H = H * alpha[:, t]
        u = beta[:, t] * (v[:, t] - (k[:, t, :, None] @ H)[:, :, 0])
        H = H + k[:, t, :, :, None] * u[:, :, None]
        outs.append((q[:, t, :, None] @ H)[:, :, 0])
    s["h"].copy_(H)
    return dict(out=torch.stack(outs, 1).to(s["v"].dtype), h=s["h"])


def _plain_bwd(s):
    _, _, c, H0, U = _plain_fwd(s, s["h0"], CHUNK)
    B, L, Hv, dv = s["v"].shape
    Hk, n, C = s["q"].shape[2], H0.shape[2], CHUNK
    dO = s["dout"].float()
    dO = torch.cat([dO, dO.new_zeros((B, n * C - L, Hv, dv))], 1) if n * C > L else dO
    dO = dO.transpose(1, 2).reshape(B, Hv, n, C, dv).contiguous()
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    dU0 = t(c["P"]) @ dO
    QdO = t(c["q"]) @ (c["e0"][..., None] * dO)
    Kb = (c["beta"] * c["e0"])[..., None] * c["k"]
    dH = s["dh_last"] if s["dh_last"] is not None else torch.zeros_like(H0[:, :, 0])
    dH1s, dRs = [None] * n, [None] * n
    for j in range(n - 1, -1, -1):
        dH1s[j] = dH
        dR = t(c["T"][:, :, j]) @ (dU0[:, :, j] + c["kC"][:, :, j] @ dH)
        dRs[j] = dR
        dH = c["aC"][:, :, j, None, None] * dH + QdO[:, :, j] - t(Kb[:, :, j]) @ dR
    dH1, dR = torch.stack(dH1s, 2), torch.stack(dRs, 2)
    beta, e0, eC = c["beta"][..., None], c["e0"][..., None], c["eC"][..., None]
    dP, dA_ = dO @ t(U), -(dR @ t(U))
    qH, kH, kU = e0 * (dO @ t(H0)), e0 * beta * (dR @ t(H0)), eC * (U @ t(dH1))
    dPM, dS = c["M"] * dP, beta * c["low"] * dA_
    dq = s["scale"] * (qH + dPM @ c["k"])
    dk = t(dPM) @ c["q"] + kU - kH + dS @ c["k"] + t(dS) @ c["k"]
    db = (dR * U).sum(-1) * (1 - c["beta"])
    # what crosses a step's decay: pairs on both sides of it, the state in and the state out
    E = dPM * c["QK"] + dS * c["S"]
    own_sum = E.sum(-1) - E.sum(-2) + (qH * c["q"]).sum(-1) - (kH * c["k"]).sum(-1) - (kU * c["k"]).sum(-1)
    own_sum[..., -1] += (kU * c["k"]).sum((-1, -2)) + c["aC"] * (dH1 * H0).sum((-1, -2))
    dg = own_sum.flip(-1).cumsum(-1).flip(-1)

    def back(x):
        return x.reshape((B, Hv, n * C) + x.shape[4:])[:, :, :L].transpose(1, 2)

    dg, db = back(dg), back(db)
    if s["reset"] is not None:
        dg = dg * (s["reset"] == 0)[..., None]
    draw_ = dg * s["A"] * torch.sigmoid(c["raw"])
    heads = lambda x: back(x).reshape(B, L, Hk, Hv // Hk, -1).sum(3)  # noqa: E731
    dt = s["v"].dtype
    return dict(dq=heads(dq).to(dt), dk=heads(dk).to(dt), dv=back(beta * dR).to(dt),
                d_dt_raw=draw_.to(dt), dbeta_raw=db.to(dt), dA=(dg * c["delta"]).sum((0, 1)),
                d_dt_bias=draw_.sum((0, 1)), dh0=dH)


def _rotate(s, x, back=False):
    """The first rot entries of x (B, L, H, d) turned by each token's angle."""
    rot = s["case"]["rot"]
    if not rot:
        return x
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    sin = -sin if back else sin
    y = x.clone()
    if s["case"]["pairs"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _norm_factor(s, x):
    sq = x.square().sum(-1, keepdim=True)
    return torch.rsqrt((sq if s["case"]["kind"] == "l2" else sq / x.shape[-1]) + s["eps"])


def _plain_norm(s, x, w):
    x32 = x.float()
    return _rotate(s, x32 * _norm_factor(s, x32) * w).to(x.dtype)


def _plain_norm_bwd(s, x, w, dy):
    x32 = x.float()
    r = _norm_factor(s, x32)
    n = x32 * r
    dz = _rotate(s, dy.float(), back=True)
    dn = dz * w
    dot = (dn * n).sum(-1, keepdim=True)
    dx = r * (dn - n * (dot if s["case"]["kind"] == "l2" else dot / x.shape[-1]))
    return dx.to(x.dtype), (dz * n).sum((0, 1, 2))


# ---- work and exact values ----

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, L = case["B"], case["L"]
    if case["op"].startswith("norm"):
        n = B * L * (case["Hq"] + case["Hk"]) * case["d"]
        table = B * L * (case["rot"] * 4 + 4 if case["rot"] else 0)
        if case["op"] == "norm":
            return dict(bytes=2 * n * e + table, flops=6.0 * n)
        return dict(bytes=3 * n * e + table, flops=14.0 * n)
    Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
    qk, vo, gates, state = 2 * B * L * Hk * dk, B * L * Hv * dv, 2 * B * L * Hv, B * Hv * dk * dv
    per = float(B * L * Hv * dk * dv)  # entries of the states that the recurrence passes through
    if case["op"] == "step":
        return dict(bytes=(qk + 2 * vo + gates) * e + 2 * 4 * state, flops=7 * per)
    marks = B * L if case["packed"] else 0
    states = 4 * state * (2 if case["state"] else 1)
    if case["op"] == "fwd":
        return dict(bytes=(qk + 2 * vo + gates) * e + states + marks, flops=7 * per)
    # state again (5), adjoint (7), gradients of q, k, the write and the decay (8)
    return dict(bytes=(2 * qk + 3 * vo + 2 * gates) * e + states + (4 * state if case["state"] else 0) + marks,
                flops=20 * per)


def exact(case, seed):
    s = prepare(case, seed)
    f = lambda x: None if x is None else x.double()  # noqa: E731
    if case["op"].startswith("norm"):
        return _exact_norm(s, case)
    B, L, Hk, dk = s["q"].shape
    Hv, dv = s["v"].shape[2:]
    head = torch.arange(Hv, device=s["v"].device) // (Hv // Hk)
    q, k, v = f(s["q"])[:, :, head] * s["scale"], f(s["k"])[:, :, head], f(s["v"])
    raw = f(s["dt_raw"]) + f(s["dt_bias"])
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    beta = torch.sigmoid(f(s["beta_raw"]))
    alpha = torch.exp(f(s["A"]) * delta)
    if s["reset"] is not None:
        alpha = alpha * (s["reset"] == 0)[..., None]
    start = s["h"] if case["op"] == "step" else s["h0"]
    H = f(start) if start is not None else q.new_zeros((B, Hv, dk, dv))
    out = q.new_empty((B, L, Hv, dv))
    keep = q.new_empty((L + 1, B, Hv, dk, dv)) if case["op"] == "bwd" else None
    for t in range(L):
        if keep is not None:
            keep[t] = H
        H = H * alpha[:, t, :, None, None]
        u = beta[:, t, :, None, None] * (v[:, t, :, None] - k[:, t, :, None] @ H)
        H = H + k[:, t, :, :, None] * u
        if keep is None:
            out[:, t] = (q[:, t, :, None] @ H)[:, :, 0]
    if case["op"] == "step":
        return dict(out=out, h=H)
    if case["op"] == "fwd":
        return dict(out=out, h_last=H)
    keep[L] = H
    do = f(s["dout"])
    dH = f(s["dh_last"]) if s["dh_last"] is not None else torch.zeros_like(H)
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dgate, db = torch.zeros_like(alpha), torch.zeros_like(beta)
    for t in range(L - 1, -1, -1):
        a, b = alpha[:, t, :, None, None], beta[:, t, :, None]
        kt, qt, dot_ = k[:, t], q[:, t], do[:, t]
        dH = dH + qt[..., :, None] * dot_[..., None, :]
        dq[:, t] = (keep[t + 1] @ dot_[..., None])[..., 0]
        before = keep[t] * a
        r = v[:, t] - (kt[..., None, :] @ before)[..., 0, :]
        du = (kt[..., None, :] @ dH)[..., 0, :]
        db[:, t] = (du * r).sum(-1)
        dr = b * du
        dv_[:, t] = dr
        dk_[:, t] = (dH @ (b * r)[..., None])[..., 0] - (before @ dr[..., None])[..., 0]
        dH = dH - kt[..., :, None] * dr[..., None, :]
        dgate[:, t] = (dH * before).sum((-1, -2))
        dH = dH * a
    per_head = lambda x: x.reshape(B, L, Hk, Hv // Hk, dk).sum(3)  # noqa: E731
    draw_ = dgate * f(s["A"]) * torch.sigmoid(raw)
    return dict(dq=per_head(dq) * s["scale"], dk=per_head(dk_), dv=dv_, d_dt_raw=draw_,
                dbeta_raw=db * beta * (1 - beta), dA=(dgate * delta).sum((0, 1)), d_dt_bias=draw_.sum((0, 1)), dh0=dH)


def _exact_norm(s, case):
    """Both directions from the norm's definition; the rotation as a product of complex numbers."""
    rot = case["rot"]
    turn = None
    if rot:
        at = s["positions"].long()
        turn = torch.complex(s["cos"].double(), s["sin"].double())[at][:, :, None]

    def pairs(x):
        if case["pairs"] == "half":
            return torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous())
        return torch.view_as_complex(x[..., :rot].contiguous().unflatten(-1, (-1, 2)))

    def turned(x, by):
        if by is None:
            return x
        z = pairs(x) * by
        first = torch.cat([z.real, z.imag], -1) if case["pairs"] == "half" else torch.view_as_real(z).flatten(-2)
        return torch.cat([first, x[..., rot:]], -1)

    def size(x):
        sq = (x * x).sum(-1, keepdim=True)
        return torch.sqrt((sq if case["kind"] == "l2" else sq / x.shape[-1]) + s["eps"])

    got = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s["w" + name].double()
        m = size(x)
        if case["op"] == "norm":
            got[name] = turned(w * x / m, turn)
            continue
        dz = turned(s["d%s_out" % name].double(), None if turn is None else turn.conj())
        got["dw" + name] = (dz * x / m).sum((0, 1, 2))
        share = 1.0 if case["kind"] == "l2" else 1.0 / x.shape[-1]
        got["d" + name] = dz * w / m - x * share * (dz * w * x).sum(-1, keepdim=True) / m ** 3
    return got

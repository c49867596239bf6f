"""Float64 oracle of the gated delta rule and of the head norms: numpy, step by
step from the definition in include/ssm_scan.h. Test infrastructure only, like
the rest of this package; it shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def _gates(dt_raw, A, beta_raw, dt_bias, reset, beta_scale):
    raw = dt_raw + (0.0 if dt_bias is None else dt_bias)
    delta = np.logaddexp(raw, 0.0)
    alpha = np.exp(A * delta)
    if reset is not None:
        alpha = np.where((reset != 0)[..., None], 0.0, alpha)
    return raw, delta, alpha, beta_scale / (1.0 + np.exp(-beta_raw))


def _per_value_head(x, Hv):
    return np.repeat(x, Hv // x.shape[2], axis=2) if x.shape[2] else x


def delta_fwd(q, k, v, dt_raw, A, beta_raw, dt_bias=None, reset=None, h0=None, scale=1.0, beta_scale=1.0,
              want_states=False):
    """(out (B,L,Hv,dv), h_last (B,Hv,dk,dv)); with want_states also the state before each step (L + 1 of them)."""
    B, L, Hv, dv = v.shape
    dk = k.shape[3]
    _, _, alpha, beta = _gates(dt_raw, A, beta_raw, dt_bias, reset, beta_scale)
    q, k = _per_value_head(q, Hv), _per_value_head(k, Hv)
    H = np.zeros((B, Hv, dk, dv)) if h0 is None else np.array(h0, np.float64)
    out, states = np.zeros((B, L, Hv, dv)), [H]
    for t in range(L):
        Hd = alpha[:, t, :, None, None] * H
        u = beta[:, t, :, None] * (v[:, t] - np.einsum("bhkv,bhk->bhv", Hd, k[:, t]))
        H = Hd + k[:, t, :, :, None] * u[:, :, None, :]
        out[:, t] = scale * np.einsum("bhkv,bhk->bhv", H, q[:, t])
        if want_states:
            states.append(H)
    return (out, H, states) if want_states else (out, H)


def delta_bwd(q, k, v, dt_raw, A, beta_raw, dout, dt_bias=None, reset=None, h0=None, dh_last=None, scale=1.0,
              beta_scale=1.0):
    """Gradients of sum dout out + sum dh_last h_last, by the chain rule step by step in reverse."""
    B, L, Hv, dv = v.shape
    Hk = k.shape[2]
    raw, delta, alpha, beta = _gates(dt_raw, A, beta_raw, dt_bias, reset, beta_scale)
    _, H, states = delta_fwd(q, k, v, dt_raw, A, beta_raw, dt_bias, reset, h0, scale, beta_scale, want_states=True)
    q, k = _per_value_head(q, Hv), _per_value_head(k, Hv)
    dH = np.zeros_like(H) if dh_last is None else np.array(dh_last, np.float64)
    dq, dk, dv_ = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dalpha, dbeta = np.zeros_like(alpha), np.zeros_like(beta)
    for t in range(L - 1, -1, -1):
        dH = dH + scale * q[:, t, :, :, None] * dout[:, t, :, None, :]
        dq[:, t] = scale * np.einsum("bhkv,bhv->bhk", states[t + 1], dout[:, t])
        Hd = alpha[:, t, :, None, None] * states[t]
        r = v[:, t] - np.einsum("bhkv,bhk->bhv", Hd, k[:, t])
        du = np.einsum("bhkv,bhk->bhv", dH, k[:, t])
        dbeta[:, t] = np.sum(du * r, -1)
        dr = beta[:, t, :, None] * du
        dv_[:, t] = dr
        dk[:, t] = (np.einsum("bhkv,bhv->bhk", dH, beta[:, t, :, None] * r) -
                    np.einsum("bhkv,bhv->bhk", Hd, dr))
        dHd = dH - k[:, t, :, :, None] * dr[:, :, None, :]
        dalpha[:, t] = np.sum(dHd * states[t], (-1, -2))
        dH = alpha[:, t, :, None, None] * dHd
    dg = dalpha * alpha
    d_dt = dg * A / (1.0 + np.exp(-raw))
    heads = lambda x: x.reshape(B, L, Hk, -1, x.shape[-1]).sum(3) if Hv else np.zeros((B, L, Hk, x.shape[-1]))  # noqa: E731
    return dict(dq=heads(dq), dk=heads(dk), dv=dv_, d_dt_raw=d_dt, dbeta_raw=dbeta * beta * (1.0 - beta / beta_scale),
                dA=(dg * delta).sum((0, 1)), d_dt_bias=d_dt.sum((0, 1)), dh0=dH)


def _turn_matrix(cos, sin, d, interleaved):
    """(tokens.., d, d) matrix of the rotation of each token."""
    half = cos.shape[-1]
    R = np.broadcast_to(np.eye(d), cos.shape[:-1] + (d, d)).copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        R[..., a, a], R[..., a, b] = cos[..., i], -sin[..., i]
        R[..., b, a], R[..., b, b] = sin[..., i], cos[..., i]
    return R


def qk_norm(x, w=None, kind="rms", eps=1e-6, cos=None, sin=None, interleaved=False, dout=None):
    """One of q, k (B,L,H,d); cos, sin (B,L,pairs) are each token's angles. Returns the
    outputs, or with dout the pair (dx, dw)."""
    d = x.shape[-1]
    w = np.ones(d) if w is None else w
    share = 1.0 if kind == "l2" else 1.0 / d
    size = np.sqrt(share * np.sum(x * x, -1, keepdims=True) + eps)
    n = x / size
    R = None if cos is None else _turn_matrix(cos, sin, d, interleaved)[:, :, None]
    if dout is None:
        y = n * w
        return y if R is None else (R @ y[..., None])[..., 0]
    dz = dout if R is None else (np.swapaxes(R, -1, -2) @ dout[..., None])[..., 0]
    dn = dz * w
    dx = dn / size - x * share * np.sum(dn * x, -1, keepdims=True) / size ** 3
    return dx, (dz * n).sum((0, 1, 2))

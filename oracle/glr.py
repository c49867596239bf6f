"""Float64 oracle of the gated linear recurrence: the definition, step by step, and its gradients.

Plain numpy, sequential in time; arrays as the library takes them (u, dt_raw, in_raw,
z (B, L, D); A and the biases (D,); reset (B, L); states (B, D)).
"""
import numpy as np


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def gates(dt_raw, A, dt_bias, in_raw, in_bias, decay, mix):
    """s, a, i, c of every step, resets not yet applied."""
    raw = dt_raw + (0.0 if dt_bias is None else dt_bias)
    s = _sigmoid(raw) if decay == "sigmoid" else np.logaddexp(0.0, raw)
    g = A * s
    a = np.exp(g)
    i = np.ones_like(raw) if in_raw is None else _sigmoid(in_raw + (0.0 if in_bias is None else in_bias))
    c = {"unit": lambda: np.sqrt(-np.expm1(2.0 * g)), "rest": lambda: -np.expm1(g), "one": lambda: np.ones_like(g)}[mix]()
    slope = s * (1.0 - s) if decay == "sigmoid" else _sigmoid(raw)
    return s, a, i, c, slope


def glr_fwd(u, dt_raw, A, dt_bias=None, in_raw=None, in_bias=None, z=None, reset=None, h0=None, decay="sigmoid",
            mix="unit", states=False):
    """(out, h_last), and the states before every step with ``states``."""
    B, L, D = u.shape
    _, a, i, c, _ = gates(dt_raw, A, dt_bias, in_raw, in_bias, decay, mix)
    h = np.zeros((B, D)) if h0 is None else np.array(h0, np.float64)
    out, before = np.empty((B, L, D)), np.empty((B, L, D))
    for t in range(L):
        before[:, t] = h
        h = a[:, t] * h + c[:, t] * i[:, t] * u[:, t]
        if reset is not None:
            h = np.where(reset[:, t, None] != 0, i[:, t] * u[:, t], h)
        out[:, t] = h
    now = out
    if z is not None:
        out = now * z * _sigmoid(z)
    return (out, h, before, now) if states else (out, h)


def glr_bwd(u, dt_raw, A, dout, dt_bias=None, in_raw=None, in_bias=None, z=None, reset=None, h0=None, dh_last=None,
            decay="sigmoid", mix="unit"):
    """Gradients of sum dout * out + sum dh_last * h_last, named as the library's."""
    B, L, D = u.shape
    s, a, i, c, slope = gates(dt_raw, A, dt_bias, in_raw, in_bias, decay, mix)
    _, _, before, now = glr_fwd(u, dt_raw, A, dt_bias, in_raw, in_bias, z, reset, h0, decay, mix, states=True)
    on = np.zeros((B, L, 1), bool) if reset is None else (reset != 0)[..., None]
    c = np.where(on, 1.0, c)
    dy, g = dout, {}
    if z is not None:
        sz = _sigmoid(z)
        g["dz"] = dout * now * sz * (1.0 + z * (1.0 - sz))
        dy = dout * z * sz
    lam = np.empty((B, L, D))
    m = np.zeros((B, D)) if dh_last is None else np.array(dh_last, np.float64)
    for t in range(L - 1, -1, -1):
        lam[:, t] = dy[:, t] + m
        m = np.where(on[:, t], 0.0, a[:, t] * lam[:, t])
    g["dh0"] = m
    g["du"] = lam * c * i
    if in_raw is not None:
        g["din_raw"] = lam * c * u * i * (1.0 - i)
        g["din_bias"] = g["din_raw"].sum((0, 1))
    if mix == "unit":
        dc = np.where(c == 0.0, 0.0, -a / np.where(c == 0.0, 1.0, c))
    else:
        dc = -np.ones_like(a) if mix == "rest" else np.zeros_like(a)
    dg = np.where(on, 0.0, lam * a * (before + i * u * dc))
    g["d_dt_raw"] = dg * A * slope
    g["d_dt_bias"] = g["d_dt_raw"].sum((0, 1))
    g["dA"] = (dg * s).sum((0, 1))
    return g

"""Float64 oracle of the norms around a block: the definitions and their gradients, in plain numpy."""
import numpy as np


def _factor(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps)


def _norm_back(v, eps, dn):
    """Gradient of v from that of v r(v)."""
    r = _factor(v, eps)
    return r * dn - v * r ** 3 * np.mean(dn * v, axis=-1, keepdims=True)


def _silu(z):
    s = 1.0 / (1.0 + np.exp(-z))
    return z * s, s * (1.0 + z * (1.0 - s))


def gated_norm(x, z, w=None, eps=1e-6, gate_first=False, dout=None):
    """The output for x, z (B, L, H, d) and w (d,) or (H, d); with dout the gradients (dx, dz, dw)."""
    one = np.ones(x.shape[-1]) if w is None else w
    gate, slope = _silu(z)
    v = x * gate if gate_first else x
    n = v * _factor(v, eps)
    if dout is None:
        return one * n if gate_first else one * n * gate
    over = (0, 1) if one.ndim == 2 else (0, 1, 2)
    if gate_first:
        dv = _norm_back(v, eps, dout * one)
        return dv * gate, dv * x * slope, (dout * n).sum(over)
    return _norm_back(x, eps, dout * one * gate), dout * one * n * slope, (dout * gate * n).sum(over)


def block_norm(y, x=None, w=None, post=False, w_post=None, gate=None, scale=1.0, eps=1e-6, dout=None, dx_out=None):
    """(out, x_out); with dout the gradients as a dict, named as the library's."""
    D = y.shape[-1]
    w, wp = (np.ones(D) if t is None else t for t in (w, w_post))
    k = scale * (np.ones(D) if gate is None else gate[:, None] if gate.ndim == 2 else gate)
    yn = y * _factor(y, eps) if post else y
    m = yn * wp if post else y
    s = k * m if x is None else x + k * m
    n = s * _factor(s, eps)
    if dout is None:
        return w * n, s
    dX = _norm_back(s, eps, dout * w) + (0.0 if dx_out is None else dx_out)
    dm = k * dX
    g = dict(dy=_norm_back(y, eps, dm * wp) if post else dm, dw=(dout * n).sum((0, 1)))
    if x is not None:
        g["dx"] = dX
    if post:
        g["dw_post"] = (dm * yn).sum((0, 1))
    if gate is not None:
        g["dgate"] = (scale * m * dX).sum(1 if gate.ndim == 2 else (0, 1))
    return g

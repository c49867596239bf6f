"""Pins of the delta-rule and head-norm oracle (oracle/delta.py): closed forms
and central differences, on the CPU."""
import numpy as np
import pytest

from oracle import delta as od


def make(seed, B=2, L=5, Hk=2, G=2, dk=3, dv=4, reset=True):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    Hv = Hk * G
    x = dict(q=n((B, L, Hk, dk)), k=n((B, L, Hk, dk)) * 0.6, v=n((B, L, Hv, dv)), dt_raw=n((B, L, Hv)),
             A=-rng.uniform(0.2, 2.0, Hv), beta_raw=n((B, L, Hv)), dt_bias=n(Hv), h0=n((B, Hv, dk, dv)))
    r = np.zeros((B, L), np.uint8)
    if reset:
        r[0, 2] = r[1, 0] = 1
    return x, r, rng


def test_full_beta_and_unit_keys_store_the_value_exactly():
    """beta = 1 and |k| = 1: after a step the state answers that key with that value."""
    x, _, _ = make(1, reset=False)
    k = x["k"] / np.linalg.norm(x["k"], axis=-1, keepdims=True)
    x.update(k=k, q=k, beta_raw=np.full_like(x["beta_raw"], 60.0))
    out, _ = od.delta_fwd(**x)
    assert np.allclose(out, x["v"], atol=1e-12)


def test_no_decay_no_correction_is_a_sum_of_outer_products():
    """A = 0 and orthonormal keys: H_t = sum beta k v^T, read out by each key."""
    L = 4
    k = np.eye(L)[None, :, None, :]
    rng = np.random.default_rng(2)
    v, b = rng.standard_normal((1, L, 1, 3)), rng.standard_normal((1, L, 1))
    out, H = od.delta_fwd(k, k, v, np.zeros((1, L, 1)), np.zeros(1), b)
    beta = 1 / (1 + np.exp(-b))
    assert np.allclose(H[0, 0], beta[0, :, 0, None] * v[0, :, 0])
    assert np.allclose(out, beta[..., None] * v)


def test_reset_starts_a_new_sequence():
    x, r, _ = make(3)
    out, H = od.delta_fwd(**x, reset=r)
    cut = {n: (a[:1, 2:] if n in ("q", "k", "v", "dt_raw", "beta_raw") else a) for n, a in x.items()}
    cut["h0"] = None
    tail, Ht = od.delta_fwd(**cut)
    assert np.allclose(out[:1, 2:], tail) and np.allclose(H[:1], Ht)


@pytest.mark.parametrize("beta_scale", [1.0, 2.0])
@pytest.mark.parametrize("reset", [False, True])
def test_gradients_against_differences(reset, beta_scale):
    x, r, rng = make(4, reset=reset)
    w = dict(reset=r if reset else None, scale=0.7, beta_scale=beta_scale)
    out, H = od.delta_fwd(**x, **w)
    dout, dh = rng.standard_normal(out.shape), rng.standard_normal(H.shape)
    g = od.delta_bwd(**x, dout=dout, dh_last=dh, **w)

    def loss(y):
        o, h = od.delta_fwd(**y, **w)
        return np.sum(o * dout) + np.sum(h * dh)

    names = dict(q="dq", k="dk", v="dv", dt_raw="d_dt_raw", A="dA", beta_raw="dbeta_raw", dt_bias="d_dt_bias", h0="dh0")
    for name, gname in names.items():
        for _ in range(6):
            i = tuple(rng.integers(0, s) for s in x[name].shape)
            lo, hi = {**x, name: x[name].copy()}, {**x, name: x[name].copy()}
            lo[name][i] -= 1e-5
            hi[name][i] += 1e-5
            num = (loss(hi) - loss(lo)) / 2e-5
            # second-order differences: truncation ~ 1e-10, rounding ~ 1e-16 |loss| / 1e-5
            assert abs(num - g[gname][i]) < 1e-7 * (1 + abs(num)), (name, i)


@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients_and_length(kind, interleaved):
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((2, 3, 2, 8)), rng.uniform(0.5, 1.5, 8)
    ang = rng.uniform(0, 6, (2, 3, 3))
    kw = dict(kind=kind, eps=1e-3, cos=np.cos(ang), sin=np.sin(ang), interleaved=interleaved)
    y = od.qk_norm(x, **kw)
    # a rotation keeps the length, which the norm fixes up to eps
    n2 = np.sum(x * x, -1)
    want = n2 / (n2 + 1e-3) if kind == "l2" else 8 * n2 / (n2 + 8e-3)
    assert np.allclose(np.sum(y * y, -1), want)
    dout = rng.standard_normal(x.shape)
    dx, dw = od.qk_norm(x, w, dout=dout, **kw)
    for name, a, g in (("x", x, dx), ("w", w, dw)):
        for _ in range(8):
            i = tuple(rng.integers(0, s) for s in a.shape)
            e = np.zeros_like(a)
            e[i] = 1e-5
            f = lambda s: np.sum(dout * od.qk_norm(x + s * e if name == "x" else x,  # noqa: E731
                                                   w + s * e if name == "w" else w, **kw))
            num = (f(1) - f(-1)) / 2e-5
            assert abs(num - g[i]) < 1e-7 * (1 + abs(num)), (name, i)

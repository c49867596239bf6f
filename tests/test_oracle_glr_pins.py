"""What pins the float64 oracle of the gated linear recurrence: closed forms, limits, the sum form, differences."""
import numpy as np
import pytest

from oracle import glr as og

KINDS = [(d, m) for d in ("sigmoid", "softplus") for m in ("unit", "rest", "one")]


def draw(seed, B=2, L=9, D=3):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    reset = np.zeros((B, L), np.uint8)
    reset[0, 4] = reset[-1, 0] = 1
    return dict(u=n((B, L, D)), dt_raw=n((B, L, D)), A=-r.uniform(0.1, 2.0, D), dt_bias=n(D), in_raw=n((B, L, D)),
                in_bias=n(D), z=n((B, L, D)), reset=reset, h0=n((B, D)))


def test_a_constant_decay_sums_a_geometric_series():
    """dt_raw = 0: a = e^(A/2); a constant input gives c u (1 - a^t) / (1 - a)."""
    A, L = np.array([-0.2, -3.0]), 12
    u = np.ones((1, L, 2))
    a = np.exp(A / 2)
    for mix, c in (("unit", np.sqrt(1 - a * a)), ("rest", 1 - a), ("one", np.ones(2))):
        out, h = og.glr_fwd(u, np.zeros((1, L, 2)), A, mix=mix)
        want = c * (1 - a[None] ** np.arange(1, L + 1)[:, None]) / (1 - a)
        assert np.allclose(out[0], want, rtol=1e-13) and np.allclose(h[0], want[-1], rtol=1e-13)


def test_softplus_with_rest_is_an_exponential_average():
    """A = -1: a = 1 - sigmoid(dt_raw), h = a h + (1 - a) u stays between its inputs and its start."""
    x = draw(1)
    out, _ = og.glr_fwd(x["u"], x["dt_raw"], -np.ones(3), h0=x["h0"], decay="softplus", mix="rest")
    f = 1 / (1 + np.exp(-x["dt_raw"]))
    h = x["h0"]
    for t in range(9):
        h = h + f[:, t] * (x["u"][:, t] - h)
        assert np.allclose(out[:, t], h, rtol=1e-12)


def test_unit_keeps_the_size_of_white_noise():
    r = np.random.default_rng(2)
    u = r.standard_normal((1, 4000, 50))
    out, _ = og.glr_fwd(u, np.zeros_like(u), np.full(50, -0.1))
    assert abs(out[0, 500:].std() - 1.0) < 0.02


@pytest.mark.parametrize("decay,mix", KINDS)
def test_the_materialised_sum(decay, mix):
    """out_t = sum over s of the decays between times c_s i_s u_s, within a document."""
    x = draw(3)
    out, _ = og.glr_fwd(decay=decay, mix=mix, **x)
    _, a, i, c, _ = og.gates(x["dt_raw"], x["A"], x["dt_bias"], x["in_raw"], x["in_bias"], decay, mix)
    silu = x["z"] / (1 + np.exp(-x["z"]))
    for b in range(2):
        for t in range(9):
            total = np.zeros(3)
            for s in range(t, -1, -1):
                between = np.prod(a[b, s + 1:t + 1], axis=0)
                first = x["reset"][b, s] != 0
                total += between * (1.0 if first else c[b, s]) * i[b, s] * x["u"][b, s]
                if first:
                    break
            else:
                total += np.prod(a[b, :t + 1], axis=0) * x["h0"][b]
            assert np.allclose(out[b, t], total * silu[b, t], rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("decay,mix", KINDS)
def test_gradients_against_differences(decay, mix):
    x = draw(4)
    r = np.random.default_rng(5)
    dout, dh = r.standard_normal((2, 9, 3)), r.standard_normal((2, 3))
    g = og.glr_bwd(dout=dout, dh_last=dh, decay=decay, mix=mix, **x)

    def loss(**kw):
        out, h = og.glr_fwd(decay=decay, mix=mix, **{**x, **kw})
        return (out * dout).sum() + (h * dh).sum()

    names = dict(u="du", dt_raw="d_dt_raw", in_raw="din_raw", z="dz", A="dA", dt_bias="d_dt_bias", in_bias="din_bias",
                 h0="dh0")
    for name, grad in names.items():
        way = r.standard_normal(x[name].shape)
        e = 1e-6
        diff = (loss(**{name: x[name] + e * way}) - loss(**{name: x[name] - e * way})) / (2 * e)
        assert abs(diff - (g[grad] * way).sum()) < 2e-7 * (1 + abs(diff)), name


def test_where_a_rounds_to_one_the_gate_gets_the_limit():
    """c = 0 exactly: d dt_raw and dA are finite, and nearby gates have gradients that tend to them."""
    u = np.ones((1, 2, 1))
    sizes = []
    for raw in (-40.0, -60.0, -80.0, -800.0):
        g = og.glr_bwd(u, np.full((1, 2, 1), raw), np.array([-0.1]), np.ones((1, 2, 1)))
        assert all(np.all(np.isfinite(v)) for v in g.values())
        sizes.append(np.abs(g["d_dt_raw"]).max())
    assert sizes[0] > sizes[1] > sizes[2] > sizes[3] == 0.0

"""What pins the float64 oracle of the norms around a block: sizes of normed rows, special cases, differences."""
import numpy as np
import pytest

from oracle import block as ob


def test_normed_rows_have_unit_mean_square():
    r = np.random.default_rng(0)
    x, z = r.standard_normal((2, 3, 2, 40)), r.standard_normal((2, 3, 2, 40))
    out = ob.gated_norm(x, z, eps=0.0, gate_first=True)
    assert np.allclose((out ** 2).mean(-1), 1.0)
    assert np.allclose(ob.gated_norm(x, z, eps=0.0), x / np.sqrt((x ** 2).mean(-1, keepdims=True)) * z / (1 + np.exp(-z)))
    # a huge gate passes the norm through (silu(z) / z -> 1)
    assert np.allclose(ob.gated_norm(x, np.full_like(x, 50.0), eps=0.0) / 50.0, ob.gated_norm(x, np.full_like(x, 50.0), eps=0.0,
                                                                                            gate_first=True))


def test_block_norm_special_cases():
    r = np.random.default_rng(1)
    y, x, g = r.standard_normal((2, 5, 30)), r.standard_normal((2, 5, 30)), r.standard_normal((2, 30))
    out, s = ob.block_norm(y, x, scale=0.0)
    assert np.array_equal(s, x) and np.allclose((out ** 2).mean(-1), 1.0, atol=1e-5)
    assert np.allclose(ob.block_norm(y, x, gate=g[0], scale=2.0)[1], x + 2.0 * g[0] * y)
    assert np.allclose(ob.block_norm(y, x, gate=g)[1][1], x[1] + g[1] * y[1])
    assert np.allclose((ob.block_norm(y, post=True, eps=0.0)[1] ** 2).mean(-1), 1.0)
    a, b = ob.block_norm(y, x, post=True, eps=0.0), ob.block_norm(7.0 * y, x, post=True, eps=0.0)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("per_head", [False, True])
def test_gated_gradients_against_differences(first, per_head):
    r = np.random.default_rng(2)
    x, z, dout = (r.standard_normal((2, 3, 4, 7)) for _ in range(3))
    w = r.standard_normal((4, 7) if per_head else 7)
    grads = ob.gated_norm(x, z, w, 1e-2, first, dout)
    for i, t in enumerate((x, z, w)):
        way, e = r.standard_normal(t.shape), 1e-6
        args = [x, z, w]
        loss = []
        for step in (e, -e):
            args[i] = t + step * way
            loss.append((ob.gated_norm(*args, 1e-2, first) * dout).sum())
        assert abs((loss[0] - loss[1]) / (2 * e) - (grads[i] * way).sum()) < 1e-7


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "row"])
@pytest.mark.parametrize("stream", [False, True])
def test_block_gradients_against_differences(post, gate, stream):
    r = np.random.default_rng(3)
    n = r.standard_normal
    a = dict(y=n((2, 3, 7)), x=n((2, 3, 7)) if stream else None, w=n(7), w_post=n(7) if post else None,
             gate=None if gate is None else n(7) if gate == "channel" else n((2, 7)))
    kw = dict(post=post, scale=0.7, eps=1e-2)
    dout, dx_out = n((2, 3, 7)), n((2, 3, 7))
    g = ob.block_norm(dout=dout, dx_out=dx_out, **a, **kw)
    for name in a:
        if a[name] is None:
            assert "d" + name not in g
            continue
        way, e, loss = n(a[name].shape), 1e-6, []
        for step in (e, -e):
            out, s = ob.block_norm(**{**a, name: a[name] + step * way}, **kw)
            loss.append((out * dout).sum() + (s * dx_out).sum())
        assert abs((loss[0] - loss[1]) / (2 * e) - (g["d" + name] * way).sum()) < 1e-7, name

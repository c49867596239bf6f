"""Non-finite inputs of the gated delta rule on the GPU: what they reach, and what a reset keeps from them."""
import numpy as np
import pytest

from oracle import delta as od
from selective_state_space_67_amd import workloads as wl

from delta_helpers import ARGS, GRAD, STATE, check, delta_inputs, host, on_device, wide

pytestmark = pytest.mark.gpu

SEQ = ("q", "k", "v", "dt_raw", "beta_raw")


def put(x, name, at, value):
    """`value` at one place of a stored input."""
    if x[name].dtype == np.uint16:
        value = wl.store(np.full(1, value), wl.BF16)[0]
    x[name][at] = value


def forward(x, **kw):
    import torch

    from selective_state_space_67_amd import ssm_delta_fwd

    t = on_device(x)
    B, L, Hv, dv = x["v"].shape
    hl = torch.full((B, Hv, x["k"].shape[3], dv), 7.0, device=t["A"].device)
    out = ssm_delta_fwd(*(t[n] for n in ARGS), dt_bias=t["dt_bias"], reset=t["reset"], h0=t["h0"], h_last=hl, **kw)
    torch.cuda.synchronize()
    return host(out), host(hl)


@pytest.mark.parametrize("dtype,L,pieces", [(wl.BF16, 16, 0), (wl.BF16, 17, 0), (wl.F32, 32, 0), (wl.F32, 33, 0),
                                            (wl.BF16, 150, 1), (wl.F32, 200, 3)])
@pytest.mark.parametrize("name", ["dt_raw", "beta_raw", "dt_bias", "A"])
def test_a_nan_gate_is_seen(name, dtype, L, pieces):
    """Either side of the length from which the sequence goes in chunks: the head is NaN from
    the token on, its state at the end too, and the other head is as always."""
    x = delta_inputs(1, L, 1, 2, 32, 24, dtype, seed=L, state=True)
    ref, rh = od.delta_fwd(**wide(x), scale=1.0)
    token = 5 if name in SEQ else 0
    put(x, name, (0, token, 1) if name in SEQ else (1,), np.nan)
    print(name, dtype, L, flush=True)
    out, hl = forward(x, scale=1.0, num_segments=pieces)
    assert np.isnan(out[:, token:, 1]).all() and np.isnan(hl[:, 1]).all()
    check(out[:, :, 0], ref[:, :, 0], STATE, "out of the other head")
    check(hl[:, 0], rh[:, 0], STATE, "h_last of the other head")


@pytest.mark.parametrize("name", ["dt_raw", "dt_bias", "A"])
def test_a_nan_gate_reaches_its_gradients(name):
    import torch

    from selective_state_space_67_amd import ssm_delta_bwd

    x = delta_inputs(1, 100, 1, 2, 32, 24, wl.F32, seed=3)
    put(x, name, (0, 5, 1) if name in SEQ else (1,), np.nan)
    t = on_device(x)
    g = ssm_delta_bwd(*(t[n] for n in ARGS), t["dout"], dt_bias=t["dt_bias"])
    torch.cuda.synchronize()
    for n in ("dA", "d_dt_bias"):
        v = host(g[n])
        assert np.isnan(v[1]) and np.isfinite(v[0]), n
    assert np.isnan(host(g["d_dt_raw"])[0, 5, 1]) and np.isfinite(host(g["d_dt_raw"])[0, :, 0]).all()


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("dtype,L,pieces", [(wl.BF16, 12, 0), (wl.F32, 30, 0), (wl.BF16, 90, 0), (wl.F32, 140, 2)])
def test_a_reset_token_needs_no_decay(dtype, L, pieces, value):
    """Where a document starts nothing is carried over, whatever the token's decay would be (a
    growing one that overflows included)."""
    x = delta_inputs(1, L, 1, 2, 32, 24, dtype, seed=L, resets=[(0, 7)], state=True)
    ref, rh = od.delta_fwd(**wide(x), reset=x["reset"], scale=1.0)
    put(x, "dt_raw", (0, 7, 0), value)
    put(x, "dt_raw", (0, 7, 1), value)
    print(dtype, L, value, flush=True)
    out, hl = forward(x, scale=1.0, num_segments=pieces)
    check(out, ref, STATE, "out")
    check(hl, rh, STATE, "h_last")


def test_a_reset_token_needs_no_decay_in_a_window_that_grows():
    """A positive A whose exponential overflows at the token that a document starts with."""
    x = delta_inputs(1, 10, 1, 1, 32, 24, wl.F32, seed=2, resets=[(0, 4)], state=True)
    x["A"][:] = 1e-3
    x["dt_raw"][0, 4] = 1e30
    ref, rh = od.delta_fwd(**wide({**x, "dt_raw": np.where(x["reset"][..., None] != 0, 0, x["dt_raw"])}),
                           reset=x["reset"], scale=1.0)
    out, hl = forward(x, scale=1.0)
    check(out, ref, STATE, "out")
    check(hl, rh, STATE, "h_last")


def test_a_reset_tokens_gate_has_no_gradient():
    """The decay of a token that starts a document is not used: whatever it is, its gradient is 0
    and it stays out of the sums for A and dt_bias."""
    import torch

    from selective_state_space_67_amd import ssm_delta_bwd

    x = delta_inputs(1, 100, 1, 2, 32, 24, wl.F32, seed=4, resets=[(0, 7), (0, 64)], state=True)
    ref = od.delta_bwd(**wide(x), dout=x["dout"].astype(np.float64), reset=x["reset"],
                       dh_last=x["dh_last"].astype(np.float64), scale=1.0)
    x["dt_raw"][0, 7, 0], x["dt_raw"][0, 64, 1] = np.nan, np.inf
    t = on_device(x)
    g = ssm_delta_bwd(*(t[n] for n in ARGS), t["dout"], dt_bias=t["dt_bias"], reset=t["reset"], h0=t["h0"],
                      dh_last=t["dh_last"], scale=1.0)
    torch.cuda.synchronize()
    for n, want in ref.items():
        check(g[n], want, GRAD, n)


RESETS = [(0, 40), (0, 75), (0, 150), (0, 200)]
PLACES = {"q": (0, 10, 0, 3), "k": (0, 10, 0, 3), "v": (0, 10, 1, 5), "dt_raw": (0, 10, 1), "beta_raw": (0, 10, 1),
          "h0": (0, 1, 3, 5)}


@pytest.mark.parametrize("dtype,L,dk,dv,pieces", [(wl.F32, 30, 32, 24, 0), (wl.F32, 100, 32, 24, 1),
                                                  (wl.BF16, 230, 64, 40, 1), (wl.BF16, 230, 64, 40, 3),
                                                  (wl.BF16, 100, 33, 21, 1), (wl.F32, 300, 160, 24, 2),
                                                  (wl.BF16, 1500, 64, 32, 20)])
@pytest.mark.parametrize("name,value", [("q", np.nan), ("k", np.nan), ("v", np.nan), ("v", np.inf), ("v", 3.4e38),
                                        ("dt_raw", np.nan), ("beta_raw", np.nan), ("h0", np.inf), ("h0", np.nan)])
def test_what_a_non_finite_value_reaches(name, value, dtype, L, dk, dv, pieces):
    """From its token on, to the end of its document: neither the tokens before it, nor other
    documents of its row, nor (of v and h0) other columns, whatever the length and the pieces."""
    if name == "v" and np.isfinite(value) and dtype == wl.BF16:
        value = 3.38e38  # the largest finite bfloat16 is 3.3895e38
    x = delta_inputs(1, L, 1, 2, dk, dv, dtype, seed=L + dk, resets=RESETS if L > 40 else [(0, 20)], state=True)
    ref, rh = od.delta_fwd(**wide(x), reset=x["reset"], scale=1.0)
    put(x, name, PLACES[name], value)
    print(name, value, dtype, L, pieces, flush=True)
    out, hl = forward(x, scale=1.0, num_segments=pieces)
    hit = np.zeros(out.shape, bool)
    token = 0 if name == "h0" else 10
    end = 40 if L > 40 else 20
    if name == "q":
        hit[:, 10] = True
    elif name == "k":
        hit[:, 10:end] = True
    else:
        columns = [PLACES[name][-1]] if name in ("v", "h0") else slice(None)
        hit[:, token:end, 1, columns] = True
    if np.isfinite(value):  # very large: float32 may or may not overflow there
        out = np.where(hit, 0.0, out)
        ref = np.where(hit, 0.0, ref)
    else:
        assert not np.isfinite(out[hit]).any()
        out, ref = np.where(hit, 0.0, out), np.where(hit, 0.0, ref)
    check(out, ref, STATE, "out elsewhere")
    check(hl, rh, STATE, "h_last")

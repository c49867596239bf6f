"""The gated linear recurrence in pieces that follow each other on the chip: every kind and pair of gates, gates that round to 0
and 1, and non-finite inputs, over several pieces (64 rows) and groups of them (1024), with their gradients."""
import numpy as np
import pytest

from oracle import glr as og
from selective_state_space_67_amd import workloads as wl

from delta_helpers import check, device, host
from glr_helpers import STATE, glr_inputs, on_device, pieces_bytes, wide
from test_glr_gpu import KINDS, compare_bwd, forward

pytestmark = pytest.mark.gpu

# documents that start at a piece's and a group's first and last row, next to each other, and in the last piece
CUTS = [(0, 63), (0, 64), (0, 700), (0, 1023), (0, 1024), (1, 1), (1, 127), (1, 128), (1, 1025), (1, 1090)]


def both_ways(x, decay, mix):
    import torch

    assert pieces_bytes(x) > 0
    t = on_device(x, device())
    bf16 = x["u"].dtype == np.uint16
    out, last = forward(x, t, decay, mix, out_dtype=torch.bfloat16 if bf16 else torch.float32)
    ref, rh = og.glr_fwd(decay=decay, mix=mix, **wide(x))
    check(out, ref, STATE, "out", bf16=bf16)
    check(last, rh, STATE, "h_last")
    compare_bwd(x, t, decay, mix, bf16)


@pytest.mark.parametrize("decay,mix", KINDS)
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
def test_kinds(decay, mix, gate, z, dtype):
    print(decay, mix, gate, z, dtype, flush=True)
    both_ways(glr_inputs(2, 1100, 66, dtype, seed=4, decay=decay, gate=gate, z=z, resets=CUTS, state=True), decay, mix)


@pytest.mark.parametrize("L", [16385, 33000])
def test_one_gate_over_ranges_of_pieces(L):
    """The form with softplus, 1 - a and an output gate over more rows than a range of groups (16384)."""
    print(L, flush=True)
    both_ways(glr_inputs(1, L, 66, wl.BF16, seed=L, decay="softplus", gate=False, z=True, resets=[(0, 16383), (0, 20000)],
                         state=True), "softplus", "rest")


@pytest.mark.parametrize("decay,mix", KINDS)
@pytest.mark.parametrize("L", [72, 1080])
def test_extreme_gates(decay, mix, L):
    """Gates that round to 0 and 1, decays that vanish or keep everything, in a walk and in pieces.

    A decay just below 1 is off by up to 2^-25, half of float32's step there. The gates repeat every 8 steps, and that error
    with them, so that over a memory of L steps it does not add up at random: a term c i u of a state is off by up to L 2^-25
    of itself, the state by as much of the sum of its terms' magnitudes, which is the state that |u| makes. The gradients'
    bounds hold over the short length (72 * 2^-25 = 2e-6); their kernels are the same for the other.
    """
    raws = np.array([-800.0, -100.0, -40.0, -20.0, 0.0, 20.0, 100.0, 800.0], np.float32)
    x = glr_inputs(1, L, 64, wl.F32, seed=1, z=True)
    x["dt_raw"] = np.broadcast_to(np.tile(raws, L // 8)[None, :, None], (1, L, 64)).copy()
    x["in_raw"] = np.ascontiguousarray(x["dt_raw"][:, ::-1])
    x["dt_bias"] = x["in_bias"] = None
    x["A"] = -np.logspace(-6, 3, 64).astype(np.float32)
    assert (pieces_bytes(x) > 0) == (L > 72)
    t = on_device(x, device())
    print(decay, mix, L, flush=True)
    got = [host(v) for v in forward(x, t, decay, mix)]
    w = wide(x)
    refs = og.glr_fwd(decay=decay, mix=mix, **w)
    most = og.glr_fwd(decay=decay, mix=mix, **{**w, "u": np.abs(w["u"])})
    for v, ref, terms, name in zip(got, refs, most, ("out", "h_last")):
        bound = STATE * (np.sqrt(np.mean(ref * ref)) + np.abs(ref)) + L * 2.0 ** -25 * np.abs(terms)
        assert np.all(np.abs(v - ref) <= bound), name
    if L == 72:
        compare_bwd(x, t, decay, mix, False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["u", "dt_raw", "in_raw", "z", "h0"])
def test_a_non_finite_input_stays_in_its_channel_and_document(name, bad):
    import torch

    B, L, D, at = 2, 2200, 66, 1100
    cuts = [70, 71, 1000, 1300]
    x = glr_inputs(B, L, D, wl.F32, seed=3, z=True, state=True, resets=[(b, c) for b in range(B) for c in cuts])
    assert pieces_bytes(x) > 0
    t = on_device(x, device())
    clean, clean_last = forward(x, t, "sigmoid", "unit")
    t[name][(0, 5) if name == "h0" else (0, at, 5)] = bad
    out, last = forward(x, t, "sigmoid", "unit")
    mask = torch.ones((B, L, D), dtype=torch.bool, device=device())
    mask[0, slice(0, 70) if name == "h0" else slice(1000, 1300), 5] = False
    assert torch.equal(out[mask], clean[mask]) and torch.equal(last, clean_last)

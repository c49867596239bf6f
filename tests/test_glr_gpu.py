"""Gated linear recurrence on the GPU against the float64 oracle: the sequence, pieces of it, the decode window and the gradients."""
import numpy as np
import pytest

from oracle import glr as og
from selective_state_space_67_amd import workloads as wl

from delta_helpers import check, device, host
from glr_helpers import GRAD, STATE, SUM, call, glr_inputs, on_device, wide

pytestmark = pytest.mark.gpu

KINDS = [(d, m) for d in ("sigmoid", "softplus") for m in ("unit", "rest", "one")]
# (B, L, D): one step and one channel, the step kernel's longest, tiles and waves that are not full, many tiles
SHAPES = [(1, 1, 1), (2, 1, 64), (1, 2, 65), (3, 8, 70), (1, 9, 3), (2, 63, 64), (1, 64, 130), (2, 127, 1), (1, 128, 64),
          (2, 129, 100), (3, 333, 70), (1, 1000, 130), (2, 2049, 64)]
RESETS = [(0, 0), (0, 5), (0, 6), (1, 1), (1, 64), (1, 100), (2, 127), (0, 128), (0, 300), (1, 2048)]


def forward(x, t, decay, mix, **kw):
    import torch

    from selective_state_space_67_amd import ssm_glr_fwd

    a, k = call(t)
    h_last = torch.empty((x["u"].shape[0], x["u"].shape[2]), device=device())
    out = ssm_glr_fwd(*a, reset=t["reset"], h0=t["h0"], h_last=h_last, decay=decay, mix=mix, **k, **kw)
    torch.cuda.synchronize()
    return out, h_last


def compare_bwd(x, t, decay, mix, bf16):
    import torch

    from selective_state_space_67_amd import ssm_glr_bwd

    a, k = call(t)
    g = ssm_glr_bwd(*a, t["dout"], reset=t["reset"], h0=t["h0"], dh_last=t["dh_last"], decay=decay, mix=mix,
                    grad_dtype=torch.bfloat16 if bf16 else torch.float32, **k)
    torch.cuda.synchronize()
    dh = None if x["dh_last"] is None else x["dh_last"].astype(np.float64)
    ref = og.glr_bwd(dout=wl.widen(x["dout"]), dh_last=dh, decay=decay, mix=mix, **wide(x))
    for n in g:
        if g[n] is None:
            assert n not in ref
            continue
        wide_out = n in ("dA", "d_dt_bias", "din_bias")
        check(g[n], ref[n], SUM if wide_out else GRAD, n, bf16=bf16 and n[:3] != "dh0" and not wide_out)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
@pytest.mark.parametrize("full", [True, False])
def test_sequence_and_gradients(shape, dtype, full):
    """Every option and none, over the sizes."""
    import torch

    B, L, D = shape
    x = glr_inputs(B, L, D, dtype, seed=sum(shape), gate=full, z=full, resets=RESETS if full else None, state=full)
    t = on_device(x, device())
    bf16 = dtype == wl.BF16
    print(shape, dtype, full, flush=True)
    out, last = forward(x, t, "sigmoid", "unit", out_dtype=torch.bfloat16 if bf16 else torch.float32)
    ref, rh = og.glr_fwd(**wide(x))
    check(out, ref, STATE, "out", bf16=bf16)
    check(last, rh, STATE, "h_last")
    compare_bwd(x, t, "sigmoid", "unit", bf16)


@pytest.mark.parametrize("decay,mix", KINDS)
@pytest.mark.parametrize("gate,z", [(True, False), (False, True)])
def test_kinds(decay, mix, gate, z):
    for L, dtype in ((5, wl.BF16), (200, wl.F32)):
        x = glr_inputs(2, L, 66, dtype, seed=L, decay=decay, gate=gate, z=z, resets=[(0, 3), (1, 150)], state=True)
        t = on_device(x, device())
        print(decay, mix, gate, z, L, flush=True)
        out, last = forward(x, t, decay, mix)
        ref, rh = og.glr_fwd(decay=decay, mix=mix, **wide(x))
        check(out, ref, STATE, "out")
        check(last, rh, STATE, "h_last")
        compare_bwd(x, t, decay, mix, False)


# lengths at the ends of pieces (64 rows), of groups of them (1024) and of ranges of groups (16384)
@pytest.mark.parametrize("L,D", [(256, 64), (300, 3), (1000, 130), (1024, 64), (1025, 65), (2049, 65), (16384, 3), (16385, 64),
                                 (70000, 64), (40000, 1)])
@pytest.mark.parametrize("cuts", [False, True])
def test_pieces(L, D, cuts):
    """Few channels, so that a sequence goes in pieces, with and without documents that start inside them and at their ends."""
    resets = [(0, 64), (0, 127), (0, 700), (0, 896), (0, 1023), (0, 20000), (0, 32768)] if cuts else None
    x = glr_inputs(1, L, D, wl.F32, seed=L + D, z=True, state=True, resets=resets)
    t = on_device(x, device())
    print(L, D, cuts, flush=True)
    out, last = forward(x, t, "sigmoid", "unit")
    ref, rh = og.glr_fwd(**wide(x))
    check(out, ref, STATE, "out")
    check(last, rh, STATE, "h_last")
    if L <= 2049 or D <= 3:
        compare_bwd(x, t, "sigmoid", "unit", False)


@pytest.mark.parametrize("L", [5, 100, 1500])
def test_every_token_a_document(L):
    """Nothing is handed from one token to the next: out = i u silu(z), no gradient of the decay, dh0 0."""
    import torch

    from selective_state_space_67_amd import ssm_glr_bwd

    x = glr_inputs(2, L, 66, wl.F32, seed=L, z=True, state=True, resets=[(b, t) for b in range(2) for t in range(L)])
    t = on_device(x, device())
    print(L, flush=True)
    out, last = forward(x, t, "sigmoid", "unit")
    ref, rh = og.glr_fwd(**wide(x))
    check(out, ref, STATE, "out")
    check(last, rh, STATE, "h_last")
    compare_bwd(x, t, "sigmoid", "unit", False)
    a, k = call(t)
    g = ssm_glr_bwd(*a, t["dout"], reset=t["reset"], h0=t["h0"], dh_last=t["dh_last"], **k)
    torch.cuda.synchronize()
    for n in ("d_dt_raw", "dA", "d_dt_bias", "dh0"):
        assert not g[n].any(), n


# 768 pieces of 32 rows and more are joined in segments of 64 (2048 rows)
@pytest.mark.parametrize("B,L,D", [(1, 24544, 64), (1, 24545, 3), (2, 28700, 66)])
@pytest.mark.parametrize("cuts", [False, True])
def test_gradients_of_long_sequences(B, L, D, cuts):
    resets = [(0, 4096), (0, 8191), (0, 20000), (1, 0), (1, 4095), (1, 24576)] if cuts else None
    x = glr_inputs(B, L, D, wl.F32, seed=L + D, state=True, resets=resets)
    print(B, L, D, cuts, flush=True)
    compare_bwd(x, on_device(x, device()), "sigmoid", "unit", False)


@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (1, 1, 1536), (5, 1, 100), (64, 1, 64), (3, 2, 65), (2, 5, 70), (1, 33, 64)])
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
def test_decode_window(B, T, D, dtype):
    import torch

    from selective_state_space_67_amd import ssm_glr_update
    from selective_state_space_67_amd.binding_glr import prepare_glr_update

    x = glr_inputs(B, T, D, dtype, seed=B + T + D, z=True, state=True)
    t = on_device(x, device())
    a, k = call(t)
    h, h2 = t["h0"].clone(), t["h0"].clone()
    print(B, T, D, dtype, flush=True)
    out = ssm_glr_update(h, *a, **k)
    again = prepare_glr_update(h2, *a, **k)
    first = again().clone()
    second = again()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    w = wide(x)
    ref, rh = og.glr_fwd(**w)
    check(out, ref, STATE, "out")
    check(h, rh, STATE, "h")
    w["h0"] = rh
    ref, rh = og.glr_fwd(**w)
    check(second, ref, STATE, "second out")
    check(h2, rh, STATE, "second h")


@pytest.mark.parametrize("pad", [0, 1, 7])
def test_slices_of_a_projection(pad):
    """Inputs side by side in one tensor, at strides and offsets of any alignment."""
    import torch

    from selective_state_space_67_amd import ssm_glr_bwd, ssm_glr_fwd, ssm_glr_update

    B, L, D = 2, 150, 70
    x = glr_inputs(B, L, D, wl.BF16, seed=pad, z=True, state=True)
    t = on_device(x, device())
    packed = torch.full((B, L, 4 * D + 2 * pad), float("nan"), device=device(), dtype=torch.bfloat16)
    s = dict(t)
    for j, n in enumerate(("u", "dt_raw", "in_raw", "z")):
        s[n] = packed[..., pad + j * D:pad + (j + 1) * D]
        s[n].copy_(t[n])
    a, k = call(t)
    b, m = call(s)
    assert torch.equal(ssm_glr_fwd(*a, **k), ssm_glr_fwd(*b, **m))
    g, f = ssm_glr_bwd(*a, t["dout"], **k), ssm_glr_bwd(*b, t["dout"], **m)
    assert all(torch.equal(g[n], f[n]) for n in g)
    one = {n: s[n][:, :1] for n in ("u", "dt_raw", "in_raw", "z")}  # every row's first token, L tokens apart
    h = t["h0"].clone()
    out = ssm_glr_update(h, one["u"], one["dt_raw"], t["A"], dt_bias=t["dt_bias"], in_raw=one["in_raw"],
                         in_bias=t["in_bias"], z=one["z"])
    torch.cuda.synchronize()
    w = {n: v[:, :1] if v is not None and v.ndim == 3 else v for n, v in wide(x).items()}
    check(out, og.glr_fwd(**w)[0], STATE, "out")


def test_extreme_gates():
    """Gates that round to 0 and 1, decays that vanish or keep everything: finite results and gradients."""
    import torch

    from selective_state_space_67_amd import ssm_glr_bwd

    raws = np.array([-800.0, -100.0, -40.0, -20.0, 0.0, 20.0, 100.0, 800.0], np.float32)
    x = glr_inputs(1, 72, 64, wl.F32, seed=1, z=True)
    x["dt_raw"] = np.broadcast_to(np.tile(raws, 9)[None, :, None], (1, 72, 64)).copy()
    x["in_raw"] = np.ascontiguousarray(x["dt_raw"][:, ::-1])
    x["dt_bias"] = x["in_bias"] = None
    x["A"] = -np.logspace(-6, 3, 64).astype(np.float32)
    t = on_device(x, device())
    for decay, mix in KINDS:
        out, last = forward(x, t, decay, mix)
        ref, rh = og.glr_fwd(decay=decay, mix=mix, **wide(x))
        check(out, ref, STATE, "out")
        check(last, rh, STATE, "h_last")
        a, k = call(t)
        g = ssm_glr_bwd(*a, t["dout"], decay=decay, mix=mix, **k)
        torch.cuda.synchronize()
        assert all(bool(torch.isfinite(v).all()) for v in g.values() if v is not None), (decay, mix)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["u", "dt_raw", "in_raw", "z", "h0", "dout", "dh_last"])
def test_a_non_finite_input_stays_in_its_channel_and_document(name, bad):
    import torch

    from selective_state_space_67_amd import ssm_glr_bwd

    cuts = [70, 71, 140, 160]
    B, D, at = 2, 66, 100
    for L in (200, 400):  # a walk, and pieces
        x = glr_inputs(B, L, D, wl.F32, seed=3, z=True, state=True, resets=[(b, c) for b in range(B) for c in cuts])
        t = on_device(x, device())
        clean, clean_last = forward(x, t, "sigmoid", "unit")
        a, k = call(t)
        kw = dict(reset=t["reset"], h0=t["h0"], dh_last=t["dh_last"], **k)
        g0 = ssm_glr_bwd(*a, t["dout"], **kw)
        where = {"h0": (0, 5), "dh_last": (0, 5)}.get(name, (0, at, 5))
        t[name][where] = bad
        lo, hi = {"h0": (0, 70), "dh_last": (160, L)}.get(name, (71, 140))
        out, last = forward(x, t, "sigmoid", "unit")
        g = ssm_glr_bwd(*a, t["dout"], **kw)
        torch.cuda.synchronize()
        mask = torch.ones((B, L, D), dtype=torch.bool, device=device())
        mask[0, lo:hi, 5] = False
        assert torch.equal(out[mask], clean[mask])
        rows = torch.ones((B, D), dtype=torch.bool, device=device())
        rows[0, 5] = name not in ("dh_last", "h0")
        assert torch.equal(last[rows], clean_last[rows])
        for n in ("du", "d_dt_raw", "din_raw", "dz"):
            assert torch.equal(g[n][mask], g0[n][mask]), n
        assert torch.equal(g["dh0"][rows], g0["dh0"][rows])
        other = torch.arange(D, device=device()) != 5
        for n in ("dA", "d_dt_bias", "din_bias"):
            assert torch.equal(g[n][other], g0[n][other]), n


def test_empty_and_repeated_calls():
    import torch

    from selective_state_space_67_amd import ssm_glr_bwd, ssm_glr_update

    x = glr_inputs(2, 0, 70, wl.F32, z=True, state=True)
    t = on_device(x, device())
    out, last = forward(x, t, "sigmoid", "unit")
    assert out.shape == (2, 0, 70) and torch.equal(last, t["h0"])
    a, k = call(t)
    g = ssm_glr_bwd(*a, t["dout"], dh_last=t["dh_last"], **k)
    torch.cuda.synchronize()
    assert torch.equal(g["dh0"], t["dh_last"]) and not g["dA"].any() and not g["din_bias"].any()
    h = t["h0"].clone()
    assert ssm_glr_update(h, *a, **k).numel() == 0 and torch.equal(h, t["h0"])
    x = glr_inputs(3, 700, 100, wl.BF16, z=True, state=True, resets=RESETS)
    t = on_device(x, device())
    a, k = call(t)
    one, two = (ssm_glr_bwd(*a, t["dout"], reset=t["reset"], h0=t["h0"], **k) for _ in range(2))
    torch.cuda.synchronize()
    assert all(torch.equal(one[n], two[n]) for n in one)
    assert torch.equal(forward(x, t, "sigmoid", "unit")[0], forward(x, t, "sigmoid", "unit")[0])


def test_gradients_against_differences():
    """A step along one direction of every input changes the loss as the gradients say (float32 inputs, the loss in float64)."""
    from selective_state_space_67_amd import ssm_glr_bwd

    x = glr_inputs(2, 90, 40, wl.F32, seed=9, z=True, state=True, resets=[(0, 30), (1, 64)])
    t = on_device(x, device())
    a, k = call(t)
    g = ssm_glr_bwd(*a, t["dout"], reset=t["reset"], h0=t["h0"], dh_last=t["dh_last"], **k)
    w, rng = wide(x), np.random.default_rng(10)
    names = dict(u="du", dt_raw="d_dt_raw", in_raw="din_raw", z="dz", A="dA", dt_bias="d_dt_bias", in_bias="din_bias", h0="dh0")
    for n, grad in names.items():
        way = rng.standard_normal(w[n].shape) * (0.01 if n == "A" else 1.0)
        loss = []
        for e in (1e-5, -1e-5):
            out, h = og.glr_fwd(**{**w, n: w[n] + e * way})
            loss.append((out * wl.widen(x["dout"])).sum() + (h * x["dh_last"]).sum())
        got, want = (host(g[grad]) * way).sum(), (loss[0] - loss[1]) / 2e-5
        # the gradient's own error, GRAD or SUM of each entry's size, adds up over the entries at random
        size = np.sqrt(np.sum((host(g[grad]) * way) ** 2))
        assert abs(got - want) < 2 * SUM * size + 1e-7 * abs(loss[0]), (n, got, want)

"""Head norms with the position rotation, and their gradients, on the GPU against the float64 oracle."""
import numpy as np
import pytest

from oracle import delta as od
from selective_state_space_67_amd import workloads as wl

from delta_helpers import NORM, NORM_DW, check, device

pytestmark = pytest.mark.gpu

# (B, L, Hq, Hk, d, rot): one token, odd sizes and counts, no rotation, all of it, the largest head
SHAPES = [(1, 1, 1, 1, 64, 64), (2, 5, 3, 1, 128, 64), (1, 70, 4, 2, 80, 40), (3, 7, 2, 2, 33, 10), (2, 9, 1, 5, 256, 256),
          (1, 4, 2, 1, 1, 0), (2, 3, 2, 1, 7, 6), (1, 6, 1, 1, 200, 24), (1, 300, 12, 4, 32, 16), (2, 2, 0, 3, 48, 48),
          (1, 5, 2, 2, 255, 254), (1, 3, 2, 2, 130, 130)]


def make(shape, dtype, seed):
    B, L, Hq, Hk, d, rot = shape
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    P = 50 + L
    ang = rng.uniform(0, 6.28, (P, rot // 2))
    return dict(q=wl.store(n((B, L, Hq, d)), dtype), k=wl.store(3 * n((B, L, Hk, d)), dtype),
                wq=rng.uniform(0.5, 1.5, d).astype(np.float32), wk=rng.uniform(0.5, 1.5, d).astype(np.float32),
                cos=np.cos(ang).astype(np.float32), sin=np.sin(ang).astype(np.float32),
                positions=rng.integers(0, P, (B, L)).astype(np.int32), dq_out=wl.store(n((B, L, Hq, d)), dtype),
                dk_out=wl.store(n((B, L, Hk, d)), dtype))


def options(x, t, shape, kind, interleaved, plain):
    """The call's keywords and the oracle's; plain: no weights, default positions."""
    turned = shape[5] > 0
    kw = dict(kind=kind, eps=1e-5, interleaved=interleaved)
    kw.update(cos=t["cos"] if turned else None, sin=t["sin"] if turned else None)
    at = np.broadcast_to(np.arange(shape[1]), shape[:2]) if plain else x["positions"]
    if not plain:
        kw.update(wq=t["wq"], wk=t["wk"], positions=t["positions"])
    ok = dict(kind=kind, eps=float(np.float32(1e-5)), interleaved=interleaved)
    if turned:
        ok.update(cos=x["cos"].astype(np.float64)[at], sin=x["sin"].astype(np.float64)[at])
    return kw, ok


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
@pytest.mark.parametrize("kind,interleaved,plain", [("rms", False, False), ("l2", True, False), ("l2", False, True)])
def test_both_directions(shape, dtype, kind, interleaved, plain):
    import torch

    from selective_state_space_67_amd import ssm_qk_norm_bwd, ssm_qk_norm_fwd

    x = make(shape, dtype, seed=sum(shape))
    t = {n: wl.to_torch(a, device()) for n, a in x.items()}
    kw, ok = options(x, t, shape, kind, interleaved, plain)
    bf16 = dtype == wl.BF16
    dt = torch.bfloat16 if bf16 else torch.float32
    print(shape, dtype, kind, flush=True)
    got = dict(zip("qk", ssm_qk_norm_fwd(t["q"], t["k"], out_dtype=dt, **kw)))
    g = ssm_qk_norm_bwd(t["q"], t["k"], t["dq_out"], t["dk_out"], grad_dtype=dt, **kw)
    torch.cuda.synchronize()
    for n in "qk":
        w = None if plain else x["w" + n].astype(np.float64)
        check(got[n], od.qk_norm(wl.widen(x[n]), w, **ok), NORM, n, bf16=bf16)
        dx, dw = od.qk_norm(wl.widen(x[n]), w, dout=wl.widen(x["d%s_out" % n]), **ok)
        # dx is a difference of two terms of its own size (their cancellation costs a few units more)
        check(g["d" + n], dx, 4 * NORM, "d" + n, bf16=bf16)
        check(g["dw" + n], dw, NORM_DW, "dw" + n)


def test_strided_slices_and_mixed_types():
    import torch

    from selective_state_space_67_amd import ssm_qk_norm_fwd

    shape = (2, 11, 2, 2, 64, 32)
    x = make(shape, wl.BF16, seed=3)
    t = {n: wl.to_torch(a, device()) for n, a in x.items()}
    kw, ok = options(x, t, shape, "rms", False, False)
    for pad in (0, 1, 4):
        packed = torch.full((2, 11, 256 + pad + 64), 9.0, device=device(), dtype=torch.bfloat16)
        q, k = packed[..., pad:pad + 128].unflatten(-1, (2, 64)), packed[..., pad + 128:pad + 256].unflatten(-1, (2, 64))
        q.copy_(t["q"])
        k.copy_(t["k"])
        got = ssm_qk_norm_fwd(q, k, **kw)  # float32 outputs of bfloat16 inputs
        torch.cuda.synchronize()
        for n, y in zip("qk", got):
            check(y, od.qk_norm(wl.widen(x[n]), x["w" + n].astype(np.float64), **ok), NORM, n)


def test_positions_outside_the_table():
    """Such a token's turned entries are NaN, the others and the other tokens are as always."""
    import torch

    from selective_state_space_67_amd import ssm_qk_norm_fwd

    shape = (1, 4, 1, 1, 32, 16)
    x = make(shape, wl.F32, seed=4)
    x["positions"][0] = [0, -1, 54, 53]  # the table has 54
    t = {n: wl.to_torch(a, device()) for n, a in x.items()}
    q, _ = ssm_qk_norm_fwd(t["q"], t["k"], cos=t["cos"], sin=t["sin"], positions=t["positions"])
    torch.cuda.synchronize()
    bad = torch.isnan(q.cpu())[0, :, 0]
    want = torch.zeros(4, 32, dtype=torch.bool)
    want[1:3, :16] = True
    assert torch.equal(bad, want)


def test_empty_and_determinism():
    import torch

    from selective_state_space_67_amd import ssm_qk_norm_bwd

    x = make((2, 0, 2, 1, 16, 8), wl.F32, seed=5)
    t = {n: wl.to_torch(a, device()) for n, a in x.items()}
    g = ssm_qk_norm_bwd(t["q"], t["k"], t["dq_out"], t["dk_out"], wq=t["wq"], wk=t["wk"], cos=t["cos"], sin=t["sin"])
    torch.cuda.synchronize()
    assert not g["dwq"].any() and not g["dwk"].any()
    x = make((2, 400, 4, 4, 64, 64), wl.BF16, seed=6)
    t = {n: wl.to_torch(a, device()) for n, a in x.items()}
    a, b = (ssm_qk_norm_bwd(t["q"], t["k"], t["dq_out"], t["dk_out"], wq=t["wq"], wk=t["wk"], cos=t["cos"],
                            sin=t["sin"]) for _ in range(2))
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a)

"""The example layer (examples/gated_delta_layer.py), and the operators inside a captured graph."""
import importlib.util
import os

import numpy as np
import pytest

from selective_state_space_67_amd import workloads as wl

from delta_helpers import ARGS, delta_inputs, device, on_device

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_trains_and_serves():
    spec = importlib.util.spec_from_file_location("gated_delta_layer", os.path.join(ROOT, "examples", "gated_delta_layer.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, gap = ex.main(steps=12, width=128)
    assert np.all(np.isfinite(losses)) and losses[-1] < losses[0]
    # one rounding of the output to bfloat16 on either side, through one more product
    assert gap < 2 ** -6


def test_forward_backward_window_and_norms_in_a_graph():
    """Captured once, replayed three times with eager work between, bit for bit the eager results."""
    import torch

    import selective_state_space_67_amd as ssm

    x = delta_inputs(2, 300, 1, 2, 64, 64, wl.BF16, seed=21, resets=[(0, 70), (1, 128)], state=True)
    t = on_device(x)
    one = on_device(delta_inputs(2, 1, 1, 2, 64, 64, wl.BF16, seed=22))
    cos = torch.randn(300, 16, device=device())
    sin = torch.randn(300, 16, device=device())
    h = t["h0"].clone()

    def work():
        h.copy_(t["h0"])
        q, k = ssm.ssm_qk_norm_fwd(t["q"], t["k"], kind="l2", cos=cos, sin=sin, out_dtype=torch.bfloat16)
        a = (q, k, t["v"], t["dt_raw"], t["A"], t["beta_raw"])
        last = torch.empty_like(h)
        out = [q, k, ssm.ssm_delta_fwd(*a, dt_bias=t["dt_bias"], reset=t["reset"], h0=t["h0"], h_last=last), last]
        g = ssm.ssm_delta_bwd(*a, t["dout"], dt_bias=t["dt_bias"], reset=t["reset"], h0=t["h0"], dh_last=t["dh_last"])
        n = ssm.ssm_qk_norm_bwd(t["q"], t["k"], q, k, kind="l2", cos=cos, sin=sin)
        steps = [ssm.ssm_delta_update(h, *(one[m] for m in ARGS), dt_bias=one["dt_bias"]) for _ in range(3)]
        return out + list(g.values()) + list(n.values()) + steps + [h]

    ref = [r.clone() for r in work()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for rep in range(3):
        _ = (got[2].float() * 0.0).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, ref)):
            assert torch.equal(a, b), (rep, i)

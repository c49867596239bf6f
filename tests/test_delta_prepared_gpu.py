"""prepare_delta_update: a decode window marshalled once and enqueued again and again."""
import pytest

from oracle import delta as od
from selective_state_space_67_amd import workloads as wl

from delta_helpers import ARGS, STATE, check, delta_inputs, on_device, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,T", [(wl.F32, 1), (wl.BF16, 3)])
def test_each_call_advances_the_state(dtype, T):
    import torch

    from selective_state_space_67_amd import ssm_delta_update
    from selective_state_space_67_amd.binding_delta import prepare_delta_update

    x = delta_inputs(2, T, 1, 2, 64, 40, dtype, seed=T, state=True)
    t = on_device(x)
    a = [t[n] for n in ARGS]
    h, other = t["h0"].clone(), t["h0"].clone()
    step = prepare_delta_update(h, *a, dt_bias=t["dt_bias"])
    ref = wide(x)
    for i in range(3):
        out = step()
        want = ssm_delta_update(other, *a, dt_bias=t["dt_bias"])
        torch.cuda.synchronize()
        y, ref["h0"] = od.delta_fwd(**ref, scale=64 ** -0.5)
        check(out, y, STATE, "out of call %d" % i)
        check(h, ref["h0"], STATE, "h after call %d" % i)
        assert torch.equal(out, want) and torch.equal(h, other)


def test_new_tokens_in_the_same_tensors():
    """The caller writes the next token's inputs into the tensors that the call was prepared with."""
    import torch

    from selective_state_space_67_amd.binding_delta import prepare_delta_update

    seq = ("q", "k", "v", "dt_raw", "beta_raw")
    x = delta_inputs(1, 4, 1, 2, 32, 24, wl.F32, seed=6)
    t = on_device(x)
    now = {n: (t[n][:, :1].clone() if n in seq else t[n]) for n in ARGS}
    h = torch.zeros(1, 2, 32, 24, device=t["A"].device)
    out = torch.empty(1, 1, 2, 24, device=h.device)
    step = prepare_delta_update(h, *(now[n] for n in ARGS), dt_bias=t["dt_bias"], out=out)
    ref, rh = od.delta_fwd(**wide(x), scale=32 ** -0.5)
    for i in range(4):
        for n in seq:
            now[n].copy_(t[n][:, i:i + 1])
        assert step() is out
        torch.cuda.synchronize()
        check(out, ref[:, i:i + 1], STATE, "out of token %d" % i)
    check(h, rh, STATE, "h")

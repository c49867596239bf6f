"""Calls with stream=: the current stream goes on allocating and writing while they wait and run."""
import pytest

from selective_state_space_67_amd import workloads as wl

from delta_helpers import ARGS, delta_inputs, on_device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["fwd", "bwd", "norm_bwd", "update"])
def test_the_current_stream_takes_none_of_a_calls_memory(name):
    import torch

    import selective_state_space_67_amd as ssm

    x = delta_inputs(1, 2000, 1, 2, 64, 64, wl.BF16, seed=3, state=True)
    t = on_device(x)
    a = [t[n] for n in ARGS]
    call = {
        "fwd": lambda **kw: [ssm.ssm_delta_fwd(*a, dt_bias=t["dt_bias"], h0=t["h0"], **kw)],
        "bwd": lambda **kw: list(ssm.ssm_delta_bwd(*a, t["dout"], dt_bias=t["dt_bias"], h0=t["h0"],
                                                   dh_last=t["dh_last"], **kw).values()),
        "norm_bwd": lambda **kw: list(ssm.ssm_qk_norm_bwd(t["q"], t["k"], t["k"], t["q"], **kw).values()),
        "update": lambda **kw: [ssm.ssm_delta_update(t["h0"].clone(), *(y[:, :3].contiguous() if y.dim() > 1 else y
                                                                       for y in a), **kw)],
    }[name]
    want = [w.clone() for w in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some milliseconds during which the call waits
    if name == "update":  # its inputs are made inside: ready before the call is
        side.synchronize()
    print(name, flush=True)
    got = call(stream=side)
    taken = []
    for size in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24, 1 << 26):
        for _ in range(4):
            taken.append(torch.empty(size, dtype=torch.uint8, device=t["A"].device).fill_(255))
    del taken
    side.synchronize()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_results_dropped_while_the_current_stream_reads_them():
    """A result used on the current stream and dropped is not handed out on the side stream before."""
    import torch

    import selective_state_space_67_amd as ssm

    t = on_device(delta_inputs(1, 300, 1, 2, 64, 64, wl.F32, seed=4))
    a = [t[n] for n in ARGS]
    want = ssm.ssm_delta_fwd(*a).sum()
    torch.cuda.synchronize()
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    got = ssm.ssm_delta_fwd(*a, stream=side)
    current.wait_stream(side)
    torch.cuda._sleep(20_000_000)
    total = got.sum()
    shape, device = got.shape, got.device
    del got
    with torch.cuda.stream(side):
        for _ in range(4):
            torch.empty(shape, device=device).fill_(9.0)
    torch.cuda.synchronize()
    assert torch.equal(total, want)

"""Whose memory a call of the gated linear recurrence or of the norms around a block allocates with stream= (the stand-ins
of test_delta_streams_cpu.py; nothing runs)."""
import pytest
import torch

from selective_state_space_67_amd import binding_block as bb
from selective_state_space_67_amd import binding_glr as bg

from test_delta_streams_cpu import watch  # noqa: F401

z = torch.zeros


def seq():
    return z(2, 70, 8), z(2, 70, 8), z(8)


CALLS = {
    "fwd": lambda s: bg.ssm_glr_fwd(*seq(), in_raw=z(2, 70, 8), z=z(2, 70, 8), stream=s),
    "update": lambda s: bg.ssm_glr_update(z(2, 8), *seq(), stream=s),
    "prepared": lambda s: bg.prepare_glr_update(z(2, 8), *seq(), stream=s)(),
    "bwd": lambda s: bg.ssm_glr_bwd(*seq(), z(2, 70, 8), in_raw=z(2, 70, 8), z=z(2, 70, 8), stream=s),
    "gated": lambda s: bb.ssm_gated_norm_fwd(z(2, 3, 2, 8), z(2, 3, 2, 8), stream=s),
    "gated_bwd": lambda s: bb.ssm_gated_norm_bwd(*[z(2, 3, 2, 8)] * 3, w=z(2, 8), stream=s),
    "block": lambda s: bb.ssm_block_norm_fwd(z(2, 3, 8), z(2, 3, 8), stream=s),
    "block_bwd": lambda s: bb.ssm_block_norm_bwd(*[z(2, 3, 8)] * 4, post=True, gate=z(2, 8), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_stream_that_uses_it(watch, name):  # noqa: F811
    side, current, lib, made, marked = watch
    got = CALLS[name](side)
    assert lib.ran == [77]
    assert made and all(stream is side for stream, _ in made)
    results = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    for t in results:
        assert (t.data_ptr(), current) in marked


class Anywhere:
    """A stream of whatever device."""
    cuda_stream = 0


@pytest.mark.parametrize("name", CALLS)
def test_tensors_in_host_memory_are_refused(name):
    """The kernels would be handed addresses that they cannot reach."""
    with pytest.raises(ValueError, match="cpu"):
        CALLS[name](None)
    with pytest.raises(ValueError, match="cpu"):
        bg.ssm_glr_update(z(2, 8), z(2, 1, 8), z(2, 1, 8), z(8), out=z(2, 1, 8), stream=Anywhere())

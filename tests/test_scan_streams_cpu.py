"""Whose memory a scan call with stream= allocates (the stand-ins of test_delta_streams_cpu.py)."""
import pytest
import torch

from selective_state_space_67_amd import binding as bd

from test_delta_streams_cpu import watch  # noqa: F401


def inputs():
    z = torch.zeros
    return z(1, 4, 70), z(1, 4, 70), z(4, 16), z(1, 70, 16), z(1, 70, 16)


def step():
    z = torch.zeros
    return z(1, 4, 16), z(1, 4), z(1, 4), z(4, 16), z(1, 16), z(1, 16)


CALLS = {
    "fwd": lambda s: bd.ssm_scan_fwd(*inputs(), stream=s),
    "wavefront": lambda s: bd.ssm_scan_fwd_wavefront(*inputs(), stream=s),
    "prepared fwd": lambda s: bd.prepare_scan(*inputs(), stream=s)(),
    "aggregate": lambda s: bd.ssm_scan_aggregate(*inputs()[:4], stream=s),
    "prepared aggregate": lambda s: bd.prepare_aggregate(*inputs()[:4], stream=s)(),
    "update": lambda s: bd.ssm_state_update(*step(), stream=s),
    "prepared update": lambda s: bd.prepare_state_update(*step(), stream=s)(),
    "bwd": lambda s: bd.ssm_scan_bwd(*inputs(), torch.zeros(1, 4, 70), conv_w=torch.zeros(4, 4), stream=s),
    "prepared bwd": lambda s: bd.prepare_scan_bwd(*inputs(), torch.zeros(1, 4, 70), conv_w=torch.zeros(4, 4),
                                                  stream=s)(),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_stream_that_uses_it(watch, name):  # noqa: F811
    side, current, lib, made, marked = watch
    got = CALLS[name](side)
    assert [getattr(s, "value", s) for s in lib.ran] == [77]
    assert made and all(stream is side for stream, _ in made)
    results = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    for t in results:
        assert t is None or (t.data_ptr(), current) in marked

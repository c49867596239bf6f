"""Whose memory a delta-rule or norm call with stream= allocates: shown with a stand-in for the
library and for torch's streams, so that nothing runs."""
import contextlib

import pytest
import torch

from selective_state_space_67_amd import binding as bd
from selective_state_space_67_amd import binding_delta as bdd


class Library:
    """Every size function asks for 4096 bytes, every call succeeds and notes its stream."""

    def __init__(self):
        self.ran = []

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            def size(params, n):
                n._obj.value = 4096
                return 0
            return size

        def call(params, *rest):
            self.ran.append(rest[-1])
            return 0
        return call


class Stream:
    cuda_stream = 77


@pytest.fixture
def watch(monkeypatch):
    """(side stream, library, [(stream it was allocated under, tensor)], {addresses marked as used on the current one})."""
    side, current, lib = Stream(), Stream(), Library()
    under, made, marked = [], [], set()

    @contextlib.contextmanager
    def on(stream):
        under.append(stream)
        yield
        under.pop()

    empty = torch.empty

    def noted(*a, **k):
        t = empty(*a, **k)
        made.append((under[-1] if under else None, t))
        return t

    monkeypatch.setattr(bd, "load_library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch, "empty", noted)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: marked.add((t.data_ptr(), s)), raising=False)
    return side, current, lib, made, marked


def inputs():
    z = torch.zeros
    return z(1, 70, 1, 8), z(1, 70, 1, 8), z(1, 70, 2, 6), z(1, 70, 2), z(2), z(1, 70, 2)


CALLS = {
    "fwd": lambda s: bdd.ssm_delta_fwd(*inputs(), stream=s),
    "update": lambda s: bdd.ssm_delta_update(torch.zeros(1, 2, 8, 6), *inputs(), stream=s),
    "prepared": lambda s: bdd.prepare_delta_update(torch.zeros(1, 2, 8, 6), *inputs(), stream=s)(),
    "bwd": lambda s: bdd.ssm_delta_bwd(*inputs(), torch.zeros(1, 70, 2, 6), stream=s),
    "norm": lambda s: bdd.ssm_qk_norm_fwd(*inputs()[:2], stream=s),
    "norm_bwd": lambda s: bdd.ssm_qk_norm_bwd(*inputs()[:2], *inputs()[:2], stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_stream_that_uses_it(watch, name):
    side, current, lib, made, marked = watch
    got = CALLS[name](side)
    assert lib.ran == [77]
    assert made and all(stream is side for stream, _ in made)
    results = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    for t in results:
        assert (t.data_ptr(), current) in marked

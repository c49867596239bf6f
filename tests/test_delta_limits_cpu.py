"""How many heads a call of the delta rule takes (host checks; nothing is launched)."""
import ctypes

import pytest

from test_delta_abi_cpu import SHAPE, delta, lib, refused, update  # noqa: F401


@pytest.mark.parametrize("batch,dv", [(1 << 20, 16), ((1 << 24) - 1, 64), ((1 << 23) - 1, 65), (20000, 50000)])
def test_many_small_states_are_no_more_than_a_launch_allows(lib, batch, dv):  # noqa: F811
    """A workgroup for every 64 columns of a head, of which a launch takes 2^24 - 1."""
    n = ctypes.c_size_t(7)
    p = delta(batch=batch, seqlen=1, key_heads=1, value_heads=1, dk=8, dv=dv)
    assert lib.ssm_delta_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0, lib.ssm_last_error()
    assert n.value == 0


@pytest.mark.parametrize("batch,dv", [(1 << 24, 64), (1 << 23, 65), (1 << 31, 16)])
def test_more_than_a_launch_allows(lib, batch, dv):  # noqa: F811
    size = dict(batch=batch, key_heads=1, value_heads=1, dk=8, dv=dv)
    n = ctypes.c_size_t(7)
    assert lib.ssm_delta_workspace_size(ctypes.byref(delta(seqlen=1, **size)), ctypes.byref(n)) == SHAPE
    refused(lib, "ssm_delta_fwd", delta(seqlen=1, **size), SHAPE, "workgroups")
    refused(lib, "ssm_delta_update", update(tokens=1, **size), SHAPE, "workgroups")

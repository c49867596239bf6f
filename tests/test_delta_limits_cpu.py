"""How many heads a call of the delta rule takes (host checks; nothing is launched)."""
import ctypes

import pytest

from test_delta_abi_cpu import SHAPE, backward, delta, lib, refused, update  # noqa: F401


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


def test_chunks_on_more_workgroups_than_a_launch_allows(lib):  # noqa: F811
    """4 workgroups for the 256 columns of a head: 2^22 heads are 2^24 of them."""
    n = ctypes.c_size_t(7)
    size = dict(seqlen=40, key_heads=1, value_heads=1, dk=8, dv=256)
    ok = lib.ssm_delta_workspace_size(ctypes.byref(delta(batch=(1 << 22) - 16, **size)), ctypes.byref(n))
    assert ok == 0 and n.value > 0, lib.ssm_last_error()
    assert lib.ssm_delta_workspace_size(ctypes.byref(delta(batch=1 << 22, **size)), ctypes.byref(n)) == SHAPE
    refused(lib, "ssm_delta_fwd", delta(batch=1 << 22, **size), SHAPE, "workgroups")
    size.update(batch=1 << 22)
    assert lib.ssm_delta_bwd_workspace_size(ctypes.byref(backward(**size)), ctypes.byref(n)) == SHAPE
    refused(lib, "ssm_delta_bwd", backward(**size), SHAPE, "workgroups")
    # 4 splits of the 256 entries of a key head's chunk
    size.update(batch=1 << 18, seqlen=1024, dk=256, dv=16)
    assert lib.ssm_delta_bwd_workspace_size(ctypes.byref(backward(**size)), ctypes.byref(n)) == SHAPE
    # pieces that the caller asks for
    assert lib.ssm_delta_workspace_size(ctypes.byref(delta(batch=1 << 18, seqlen=2560, key_heads=1, value_heads=1,
                                                           dk=256, dv=16, num_segments=1000)), ctypes.byref(n)) == SHAPE

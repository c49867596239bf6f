"""How many rows a scan call takes (host checks; nothing is launched): a launch's threads are counted in 32 bits."""
import ctypes

import pytest

from selective_state_space_67_amd import binding as bd

from test_abi_cpu import bwd_params, lib, scan_params  # noqa: F401

SHAPE = 2
MOST = 1 << 24  # workgroups of 256 threads that are one too many


def size(lib, fn, p):  # noqa: F811
    n = ctypes.c_size_t(0)
    return getattr(lib, fn)(ctypes.byref(p), ctypes.byref(n))


def far_apart(p):
    """Disjoint addresses for tensors of up to 2^38 bytes."""
    for i, name in enumerate(("u", "dt_raw", "z", "Bm", "Cm", "A", "dt_bias", "Dskip", "out")):
        setattr(p, name, (i + 1) << 38)
    return p


# 16 channels a workgroup up to 16 states, 8 of 512 threads for 128
@pytest.mark.parametrize("dstate,dim,most", [(16, 16, MOST), (128, 8, MOST // 2), (64, 8, MOST // 2)])
def test_real_scan(lib, dstate, dim, most):  # noqa: F811
    kw = dict(dim=dim, dstate=dstate, seqlen=1)
    for fn in ("ssm_scan_workspace_size", "ssm_scan_aggregate_workspace_size"):
        assert size(lib, fn, scan_params(batch=most - 1, **kw)) == 0, lib.ssm_last_error()
        assert size(lib, fn, scan_params(batch=most, **kw)) == SHAPE
    assert lib.ssm_scan_fwd(ctypes.byref(far_apart(scan_params(batch=most, **kw))), None) == SHAPE
    assert b"workgroups" in lib.ssm_last_error()


def test_complex_scan(lib):  # noqa: F811
    kw = dict(dim=1, dstate=16, seqlen=1, state_kind=bd.SSM_STATE_COMPLEX)
    assert size(lib, "ssm_scan_workspace_size", scan_params(batch=MOST - 1, **kw)) == 0, lib.ssm_last_error()
    assert size(lib, "ssm_scan_workspace_size", scan_params(batch=MOST, **kw)) == SHAPE


def test_backward(lib):  # noqa: F811
    for cplx in (False, True):
        p = bwd_params(cplx)
        p.batch, p.dim, p.seqlen, p.dstate = MOST, 1, 1, 16
        assert size(lib, "ssm_scan_bwd_workspace_size", p) == SHAPE
        p.batch //= 4  # the conv stage's backward: a workgroup a row and 1024 steps
        assert size(lib, "ssm_scan_bwd_workspace_size", p) == 0, lib.ssm_last_error()
        p.conv_w, p.conv_width, p.seqlen = 0x10000, 4, 4000
        assert size(lib, "ssm_scan_bwd_workspace_size", p) == SHAPE


def test_wavefront(lib):  # noqa: F811
    """A wave a channel: 4 channels a workgroup."""
    p = far_apart(scan_params(batch=MOST // 2, dim=8, seqlen=1, dstate=16))
    assert size(lib, "ssm_scan_workspace_size", p) == 0
    assert lib.ssm_scan_fwd_wavefront(ctypes.byref(p), None) == SHAPE

"""The largest launches of the block norm with a gate for each sequence; host-side checks, no GPU needed."""
import ctypes

import pytest

from test_block_abi_cpu import block
from test_delta_abi_cpu import ALIGN, SHAPE, lib, refused  # noqa: F401


@pytest.mark.parametrize("batch,dim,status", [(8191, 16384, 0), (8192, 16384, SHAPE), (16383, 8192, 0), (16384, 8192, SHAPE),
                                              (65536, 2016, 0), (65536, 2017, SHAPE)])
def test_sums_of_many_gates(lib, batch, dim, status):  # noqa: F811
    """32 sums of dgate a workgroup of 1024 threads: 2^22 workgroups are refused, fewer are not, whatever the weights'
    sums need besides (those go in launches of their own then)."""
    n = ctypes.c_size_t()
    for post in (0, 1):
        p = block(batch=batch, seqlen=1, dim=dim, gate_rows=1, post=post, w_post=None, dw_post=None)
        assert lib.ssm_block_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == status
        if status != 0:
            refused(lib, "ssm_block_norm_bwd", p, SHAPE, "workgroups")
        else:
            assert n.value == 3 * batch * dim * 4


@pytest.mark.parametrize("batch,dim,status", [(8192, 16384, ALIGN), ((1 << 22) - 1, 64, ALIGN), (1 << 22, 64, SHAPE)])
def test_a_forward_is_not_refused_for_sums_that_it_does_not_make(lib, batch, dim, status):  # noqa: F811
    """(A misaligned pointer stops what passes the checks of sizes, so that nothing runs.)"""
    refused(lib, "ssm_block_norm_fwd", block(batch=batch, seqlen=1, dim=dim, gate_rows=1, x=0x50000002), status)

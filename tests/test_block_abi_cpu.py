"""Host-side checks of the norms around a block; no GPU needed.

Fake, aligned, disjoint addresses: every call fails its checks or is an empty
problem without outputs, so nothing is launched.
"""
import ctypes

import pytest

from selective_state_space_67_amd import binding as bd
from selective_state_space_67_amd import binding_block as bb

from test_delta_abi_cpu import ALIAS, ALIGN, DTYPE, NULL, SHAPE, UNSUP, WORK, fill, lib, put, refused  # noqa: F401

GATED = ("x", "z", "w", "out", "dout", "dx", "dz", "dw", "workspace")
BLOCK = ("y", "x", "w", "w_post", "gate", "out", "x_out", "dout", "dx_out", "dy", "dx", "dw", "dw_post", "dgate", "workspace")


def gated(**kw):
    p = bb.GatedNormParams(batch=2, seqlen=5, heads=3, head_dim=32, in_dtype=bd.SSM_BF16, out_dtype=bd.SSM_F32, eps=1e-6)
    fill(p, GATED)
    p.workspace_bytes = 1 << 20
    return put(p, kw)


def block(**kw):
    p = bb.BlockNormParams(batch=2, seqlen=5, dim=96, in_dtype=bd.SSM_BF16, out_dtype=bd.SSM_F32, res_dtype=bd.SSM_F32,
                           eps=1e-6, scale=1.0, post=1)
    fill(p, BLOCK)
    p.workspace_bytes = 1 << 20
    return put(p, kw)


def both(make):
    name = "ssm_gated_norm" if make is gated else "ssm_block_norm"
    return name + "_fwd", name + "_bwd"


def test_struct_sizes(lib):  # noqa: F811
    for which, struct in bb.STRUCTS.items():
        assert lib.ssm_abi_struct_size(which) == ctypes.sizeof(struct)


@pytest.mark.parametrize("fn,make,names", [
    ("ssm_gated_norm_fwd", gated, ("x", "z", "out")), ("ssm_gated_norm_bwd", gated, ("x", "z", "dout", "dx", "dz")),
    ("ssm_block_norm_fwd", block, ("y", "out")), ("ssm_block_norm_bwd", block, ("y", "dout", "dy")),
])
def test_required_pointers(lib, fn, make, names):  # noqa: F811
    assert getattr(lib, fn)(None, None) == NULL
    for name in names:
        refused(lib, fn, make(**{name: None}), NULL, name)


SIZES = [(gated, kw) for kw in (dict(batch=-1), dict(seqlen=-1), dict(seqlen=1 << 27), dict(heads=-1), dict(heads=65537),
                                dict(head_dim=0), dict(head_dim=16385), dict(x_stride=95), dict(z_stride=-1),
                                dict(z_stride=2 ** 60), dict(batch=2 ** 55))]
SIZES += [(block, kw) for kw in (dict(batch=-1), dict(seqlen=-1), dict(seqlen=1 << 27), dict(dim=0), dict(dim=16385),
                                 dict(y_stride=95), dict(y_stride=-1), dict(y_stride=2 ** 60), dict(batch=2 ** 55),
                                 dict(gate_rows=1, batch=1 << 22))]


def named(v):
    return v.__name__ if callable(v) else str(v)


@pytest.mark.parametrize("make,kw", SIZES, ids=named)
def test_sizes(lib, make, kw):  # noqa: F811
    n = ctypes.c_size_t()
    for fn in both(make):
        refused(lib, fn, make(**kw), SHAPE)
    size = getattr(lib, both(make)[1] + "_workspace_size")
    assert size(ctypes.byref(make(**kw)), ctypes.byref(n)) == SHAPE and size(None, ctypes.byref(n)) == NULL


def test_sums_of_many_weights(lib):  # noqa: F811
    """A weight for each head: one launch sums them, 32 a workgroup of 1024 threads; 2^22 of those are refused, one less is not."""
    n = ctypes.c_size_t()
    for kw, status in ((dict(heads=8192, head_dim=16384), SHAPE), (dict(heads=8191, head_dim=16384), 0),
                       (dict(heads=65536, head_dim=2017), SHAPE), (dict(heads=65536, head_dim=2016), 0)):
        p = gated(w_per_head=1, **kw)
        assert lib.ssm_gated_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == status, kw
        if status != 0:
            refused(lib, "ssm_gated_norm_bwd", p, SHAPE, "workgroups")
        p.w_per_head = 0
        assert lib.ssm_gated_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0


def test_types_and_flags(lib):  # noqa: F811
    for make in (gated, block):
        for fn in both(make):
            refused(lib, fn, make(in_dtype=2), DTYPE)
            refused(lib, fn, make(out_dtype=-1), DTYPE)
    for fn in both(block):
        refused(lib, fn, block(res_dtype=2), DTYPE)
        refused(lib, fn, block(post=2), UNSUP, "post")
        refused(lib, fn, block(gate_rows=-1), UNSUP, "gate_rows")
    for fn in both(gated):
        refused(lib, fn, gated(gate_first=2), UNSUP, "gate_first")
        refused(lib, fn, gated(w_per_head=3), UNSUP, "w_per_head")


def test_options_that_are_off(lib):  # noqa: F811
    for fn in both(block):
        refused(lib, fn, block(post=0), UNSUP, "w_post")
        refused(lib, fn, block(gate_rows=1, gate=None), NULL, "gate")
    refused(lib, "ssm_block_norm_bwd", block(post=0, w_post=None), UNSUP, "dw_post")
    refused(lib, "ssm_block_norm_bwd", block(gate=None), NULL, "dgate")
    refused(lib, "ssm_block_norm_bwd", block(x=None), NULL, "dx")


def test_alignment(lib):  # noqa: F811
    for name in ("x", "z"):
        refused(lib, "ssm_gated_norm_fwd", gated(**{name: 0x50000001}), ALIGN, name)
    refused(lib, "ssm_gated_norm_fwd", gated(w=0x50000002), ALIGN, "w")
    refused(lib, "ssm_gated_norm_bwd", gated(dx=0x50000002), ALIGN, "dx")
    refused(lib, "ssm_gated_norm_bwd", gated(workspace=0x50000004), ALIGN, "workspace")
    refused(lib, "ssm_block_norm_fwd", block(y=0x50000001), ALIGN, "y")
    for name in ("x", "w", "w_post", "gate", "x_out"):
        refused(lib, "ssm_block_norm_fwd", block(**{name: 0x50000002}), ALIGN, name)
    for name in ("dx_out", "dx", "dw", "dw_post", "dgate"):
        refused(lib, "ssm_block_norm_bwd", block(**{name: 0x50000002}), ALIGN, name)


def test_overlaps(lib):  # noqa: F811
    g, b = gated(), block()
    refused(lib, "ssm_gated_norm_fwd", gated(out=g.z), ALIAS, "out overlaps z")
    refused(lib, "ssm_gated_norm_fwd", gated(x_stride=4000, out=g.x + 2 * 9 * 4000), ALIAS, "out overlaps x")
    refused(lib, "ssm_gated_norm_bwd", gated(dx=g.dout), ALIAS)
    refused(lib, "ssm_gated_norm_bwd", gated(dz=g.dx), ALIAS)
    refused(lib, "ssm_gated_norm_bwd", gated(workspace=g.dw), ALIAS)
    refused(lib, "ssm_block_norm_fwd", block(x_out=b.x), ALIAS, "x_out overlaps x")
    refused(lib, "ssm_block_norm_fwd", block(out=b.x_out), ALIAS)
    refused(lib, "ssm_block_norm_bwd", block(dx=b.dx_out), ALIAS)
    refused(lib, "ssm_block_norm_bwd", block(dw=b.dgate), ALIAS)


def test_workspace(lib):  # noqa: F811
    n = ctypes.c_size_t()
    for make in (gated, block):
        fn = both(make)[1]
        assert getattr(lib, fn + "_workspace_size")(ctypes.byref(make()), ctypes.byref(n)) == 0 and n.value > 0
        refused(lib, fn, make(workspace_bytes=n.value - 1), WORK)
        refused(lib, fn, make(workspace=None), WORK)


def test_empty_problems_need_no_pointers(lib):  # noqa: F811
    for kw in (dict(batch=0), dict(seqlen=0), dict(heads=0)):
        assert lib.ssm_gated_norm_fwd(ctypes.byref(gated(**dict.fromkeys(GATED), **kw)), None) == 0
        assert lib.ssm_gated_norm_bwd(ctypes.byref(gated(**dict.fromkeys(GATED), **kw)), None) == 0
    for kw in (dict(batch=0, gate_rows=1), dict(seqlen=0)):
        assert lib.ssm_block_norm_fwd(ctypes.byref(block(**dict.fromkeys(BLOCK), **kw)), None) == 0
        assert lib.ssm_block_norm_bwd(ctypes.byref(block(**dict.fromkeys(BLOCK), **kw)), None) == 0


def test_binding_refusals():
    """What the binding itself checks, before any call."""
    import torch

    z = torch.zeros
    x, y = z(2, 3, 2, 8), z(2, 3, 16)
    bb._gated(x, x, z(8))
    assert bb._gated(x, x, z(2, 8))[3] == 1
    for bad in ((x, z(2, 3, 2, 9), None), (x, x, z(9)), (x, x, z(3, 8)), (y, y, None), (x, x.transpose(1, 2), None)):
        with pytest.raises(ValueError):
            bb._gated(*bad)
    with pytest.raises(TypeError):
        bb._gated(x, x.bfloat16(), None)
    ok = dict(y=y, x=y, w=None, post=True, w_post=z(16), gate=None, res_dtype=None)
    make = lambda **kw: bb._block(**{**ok, **kw})  # noqa: E731
    make()
    assert make(gate=z(2, 16))[1][1] == 1 and make(x=y.bfloat16())[1][0] == bd.SSM_BF16
    for bad in (dict(x=z(2, 3, 17)), dict(w=z(15)), dict(gate=z(3, 16)), dict(post=False), dict(y=z(6, 16)),
                dict(x=z(2, 3, 32)[..., ::2]), dict(y=z(2, 3, 32)[..., ::2])):
        with pytest.raises(ValueError):
            make(**bad)
    for bad in (dict(w=z(16).double()), dict(x=y.bfloat16(), res_dtype=torch.float32), dict(x=None, res_dtype=torch.float16),
                dict(gate=z(16).half())):
        with pytest.raises(TypeError):
            make(**bad)


@pytest.mark.parametrize("which", bb.STRUCTS)
def test_packed_fields_are_the_structs(which):
    """Every field in its place, whatever its type."""
    fields = bb.STRUCTS[which]._fields_
    got = bb.STRUCTS[which].from_buffer_copy(bb._PACKED[which].pack(*range(1, len(fields) + 1)))
    assert [getattr(got, n) for n, _ in fields] == list(range(1, len(fields) + 1))

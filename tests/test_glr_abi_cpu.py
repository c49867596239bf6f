"""Host-side checks of the gated linear recurrence's entry points; no GPU needed.

Fake, aligned, disjoint addresses: every call fails its checks or is an empty
problem without outputs, so nothing is launched.
"""
import ctypes

import pytest

from selective_state_space_67_amd import binding as bd
from selective_state_space_67_amd import binding_glr as bg

from test_delta_abi_cpu import ALIAS, ALIGN, DTYPE, NULL, SHAPE, UNSUP, WORK, fill, lib, put, refused  # noqa: F401

PTRS = ("u", "dt_raw", "in_raw", "z", "A", "dt_bias", "in_bias", "reset", "h0", "out", "h_last", "dout", "dh_last", "du",
        "d_dt_raw", "din_raw", "dz", "dA", "d_dt_bias", "din_bias", "dh0", "workspace")


def seq(**kw):
    p = bg.GlrParams(batch=2, seqlen=70, dim=24, in_dtype=bd.SSM_BF16, out_dtype=bd.SSM_F32)
    fill(p, PTRS)
    p.workspace_bytes = 1 << 20
    return put(p, kw)


def window(**kw):
    p = bg.GlrUpdateParams(batch=2, tokens=3, dim=24, in_dtype=bd.SSM_BF16, out_dtype=bd.SSM_F32)
    fill(p, ("h", "u", "dt_raw", "in_raw", "z", "A", "dt_bias", "in_bias", "out"))
    return put(p, kw)


ALL = [("ssm_glr_fwd", seq), ("ssm_glr_bwd", seq), ("ssm_glr_update", window)]


def test_struct_sizes(lib):  # noqa: F811
    for which, struct in bg.STRUCTS.items():
        assert lib.ssm_abi_struct_size(which) == ctypes.sizeof(struct)


@pytest.mark.parametrize("fn,make,names", [
    ("ssm_glr_fwd", seq, ("u", "dt_raw", "A", "out")),
    ("ssm_glr_bwd", seq, ("u", "dt_raw", "A", "dout", "du", "d_dt_raw", "din_raw", "dz", "dA")),
    ("ssm_glr_update", window, ("h", "u", "dt_raw", "A", "out")),
])
def test_required_pointers(lib, fn, make, names):  # noqa: F811
    assert getattr(lib, fn)(None, None) == NULL
    for name in names:
        refused(lib, fn, make(**{name: None}), NULL, name)
    refused(lib, fn, make(in_raw=None), NULL, "in_bias")


def test_gradients_without_their_input(lib):  # noqa: F811
    refused(lib, "ssm_glr_bwd", seq(in_raw=None, in_bias=None), NULL, "din_raw")
    refused(lib, "ssm_glr_bwd", seq(z=None), NULL, "dz")


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(dim=-1), dict(dim=(1 << 24) + 1), dict(u_stride=23), dict(dt_stride=-1),
                                dict(in_stride=1), dict(z_stride=2 ** 60), dict(batch=2 ** 50), dict(batch=2 ** 40, dim=2 ** 24)],
                         ids=str)
def test_sizes(lib, kw):  # noqa: F811
    for fn, make in ALL:
        refused(lib, fn, make(**kw), SHAPE)
    n = ctypes.c_size_t()
    for fn in ("ssm_glr_workspace_size", "ssm_glr_bwd_workspace_size"):
        assert getattr(lib, fn)(ctypes.byref(seq(**kw)), ctypes.byref(n)) == SHAPE
        assert getattr(lib, fn)(None, ctypes.byref(n)) == NULL


def test_lengths_kinds_and_types(lib):  # noqa: F811
    for fn in ("ssm_glr_fwd", "ssm_glr_bwd"):
        refused(lib, fn, seq(seqlen=1 << 27), SHAPE)
        refused(lib, fn, seq(seqlen=-1), SHAPE)
    refused(lib, "ssm_glr_update", window(tokens=-1), SHAPE)
    for fn, make in ALL:
        refused(lib, fn, make(in_dtype=2), DTYPE)
        refused(lib, fn, make(out_dtype=-1), DTYPE)
        refused(lib, fn, make(decay=2), UNSUP, "decay")
        refused(lib, fn, make(mix=3), UNSUP, "mix")


def test_alignment(lib):  # noqa: F811
    for fn, make in ALL:
        for name in ("u", "dt_raw", "in_raw", "z"):
            refused(lib, fn, make(**{name: 0x50000001}), ALIGN, name)
        for name in ("A", "dt_bias", "in_bias"):
            refused(lib, fn, make(**{name: 0x50000002}), ALIGN, name)
    for name in ("h0", "h_last", "out"):
        refused(lib, "ssm_glr_fwd", seq(**{name: 0x50000002}), ALIGN, name)
    for name in ("h0", "dh_last", "du", "dA", "d_dt_bias", "din_bias", "dh0"):
        refused(lib, "ssm_glr_bwd", seq(**{name: 0x50000002}), ALIGN, name)
    refused(lib, "ssm_glr_update", window(h=0x50000002), ALIGN, "h")
    refused(lib, "ssm_glr_bwd", seq(workspace=0x50000080), ALIGN, "workspace")


def test_overlaps(lib):  # noqa: F811
    s = seq()
    refused(lib, "ssm_glr_fwd", seq(out=s.u), ALIAS, "out overlaps u")
    refused(lib, "ssm_glr_fwd", seq(h_last=s.h0), ALIAS)
    refused(lib, "ssm_glr_fwd", seq(h_last=s.out), ALIAS)
    # a strided input reaches past its dense size
    refused(lib, "ssm_glr_fwd", seq(z_stride=4000, out=s.z + 2 * 139 * 4000), ALIAS, "out overlaps z")
    refused(lib, "ssm_glr_bwd", seq(du=s.dout), ALIAS)
    refused(lib, "ssm_glr_bwd", seq(dz=s.din_raw), ALIAS)
    refused(lib, "ssm_glr_bwd", seq(workspace=s.dh0 & ~255), ALIAS)
    refused(lib, "ssm_glr_update", window(out=window().h), ALIAS)
    refused(lib, "ssm_glr_update", window(h=window().A), ALIAS)


def test_workspace(lib):  # noqa: F811
    n = ctypes.c_size_t(7)
    for L in (1, 70):
        assert lib.ssm_glr_workspace_size(ctypes.byref(seq(seqlen=L)), ctypes.byref(n)) == 0 and n.value == 0
    assert lib.ssm_glr_workspace_size(ctypes.byref(seq(seqlen=9000)), ctypes.byref(n)) == 0 and n.value > 0
    for kw in (dict(workspace_bytes=n.value - 1), dict(workspace=None)):
        refused(lib, "ssm_glr_fwd", seq(seqlen=9000, **kw), WORK)
    assert lib.ssm_glr_bwd_workspace_size(ctypes.byref(seq()), ctypes.byref(n)) == 0 and n.value >= 32 * 2 * 2 * 24
    for kw in (dict(workspace_bytes=n.value - 1), dict(workspace=None)):
        refused(lib, "ssm_glr_bwd", seq(**kw), WORK)


def test_more_than_a_launch_allows(lib):  # noqa: F811
    n = ctypes.c_size_t()
    ok = lambda **kw: lib.ssm_glr_workspace_size(ctypes.byref(seq(dim=1, **kw)), ctypes.byref(n))  # noqa: E731
    assert ok(batch=(1 << 26) - 1, seqlen=1) == 0
    assert ok(batch=1 << 26, seqlen=1) == SHAPE
    refused(lib, "ssm_glr_update", window(batch=1 << 26, tokens=1, dim=1), SHAPE, "workgroups")
    # 512 threads a piece, and none of the sizes is multiplied past 64 bits
    assert ok(batch=(1 << 23) - 1, seqlen=128) == 0
    assert ok(batch=1 << 23, seqlen=128) == SHAPE
    # pieces of a chain, 256 threads each; where they are too many, a walk (which has no workspace)
    assert ok(batch=7, seqlen=(1 << 27) - 1) == 0 and n.value > 0
    assert ok(batch=65, seqlen=(1 << 27) - 1) == 0 and n.value == 0
    assert ok(batch=128, seqlen=1 << 23) == 0 and n.value == 0
    assert lib.ssm_glr_bwd_workspace_size(ctypes.byref(seq(batch=1 << 20, seqlen=1 << 20, dim=1)), ctypes.byref(n)) == SHAPE
    assert lib.ssm_glr_bwd_workspace_size(ctypes.byref(seq(batch=1 << 57, seqlen=1, dim=1)), ctypes.byref(n)) == SHAPE


def test_empty_problems_need_no_pointers(lib):  # noqa: F811
    none = dict.fromkeys(PTRS)
    for kw in (dict(batch=0), dict(dim=0), dict(seqlen=0)):
        assert lib.ssm_glr_fwd(ctypes.byref(seq(**none, **kw)), None) == 0
    assert lib.ssm_glr_bwd(ctypes.byref(seq(**none, dim=0)), None) == 0
    none = dict.fromkeys(("h", "u", "dt_raw", "in_raw", "z", "A", "dt_bias", "in_bias", "out"))
    for kw in (dict(batch=0), dict(dim=0), dict(tokens=0)):
        assert lib.ssm_glr_update(ctypes.byref(window(**none, **kw)), None) == 0


def test_binding_refusals():
    """What the binding itself checks, before any call: shapes, layout, types, kinds."""
    import torch

    z = torch.zeros
    u = z(2, 5, 8)
    ok = dict(u=u, dt_raw=u, A=z(8), dt_bias=None, in_raw=u, in_bias=None, z=None, decay="sigmoid", mix="unit")
    check = lambda **kw: bg._inputs(**{**ok, **kw})  # noqa: E731
    check()
    for bad in (dict(dt_raw=z(2, 5, 9)), dict(A=z(9)), dict(u=u.transpose(1, 2)), dict(z=z(2, 5, 16)[..., ::2]),
                dict(in_raw=z(4, 5, 8)[::2]), dict(u=z(2, 1, 8).expand(2, 5, 8)), dict(in_raw=None, in_bias=z(8)),
                dict(decay="tanh"), dict(mix="full"), dict(in_bias=z(3))):
        with pytest.raises(ValueError):
            check(**bad)
    for bad in (dict(A=z(8, dtype=torch.float64)), dict(dt_raw=u.bfloat16()), dict(dt_bias=z(8).half())):
        with pytest.raises(TypeError):
            check(**bad)
    packed = z(2, 5, 40)
    assert bg._tokens(packed[..., 3:11], (2, 5, 8), "u", torch.float32) == 40
    assert bg._tokens(packed[:, :1, 3:11], (2, 1, 8), "u", torch.float32) == 200
    with pytest.raises(ValueError):
        bg._one_device(u, type("T", (), dict(get_device=lambda self: 0, device="cuda:0"))())


@pytest.mark.parametrize("which", bg.STRUCTS)
def test_packed_fields_are_the_structs(which):
    """Every field in its place, whatever its type."""
    fields = bg.STRUCTS[which]._fields_
    got = bg.STRUCTS[which].from_buffer_copy(bg._PACKED[which].pack(*range(1, len(fields) + 1)))
    assert [getattr(got, n) for n, _ in fields] == list(range(1, len(fields) + 1))

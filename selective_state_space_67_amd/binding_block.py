"""ctypes binding of the norms around a block (include/ssm_scan.h).

Argument marshalling only, as in binding.py. A mixer's output, its gate and a block's
output may be slices of one packed tensor: entries are dense inside a token, tokens lie a
fixed stride apart, batch rows follow each other. Everything else is contiguous.

Streams as in binding.py: what a call allocates belongs to the stream that it runs on.
"""
from __future__ import annotations

import ctypes

from . import binding as _b
from .binding_delta import _need
from .binding_delta import _tokens as _head_tokens
from .binding_glr import _at, _call, _new, _one_device, _space, _sum, _tokens, check_layouts, packer

_i64, _i32, _vp, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float


class GatedNormParams(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("heads", _i64), ("head_dim", _i64), ("in_dtype", _i32),
                ("out_dtype", _i32), ("x", _vp), ("z", _vp), ("x_stride", _i64), ("z_stride", _i64), ("w", _vp),
                ("out", _vp), ("dout", _vp), ("dx", _vp), ("dz", _vp), ("dw", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("eps", _f32), ("gate_first", _i32), ("w_per_head", _i32),
                ("reserved0", _i32)]


class BlockNormParams(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("dim", _i64), ("in_dtype", _i32), ("out_dtype", _i32),
                ("res_dtype", _i32), ("gate_rows", _i32), ("y", _vp), ("y_stride", _i64), ("x", _vp), ("w", _vp),
                ("w_post", _vp), ("gate", _vp), ("out", _vp), ("x_out", _vp), ("dout", _vp), ("dx_out", _vp),
                ("dy", _vp), ("dx", _vp), ("dw", _vp), ("dw_post", _vp), ("dgate", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("eps", _f32), ("scale", _f32), ("post", _i32),
                ("reserved0", _i32)]


STRUCTS = {10: GatedNormParams, 11: BlockNormParams}
_PACKED = {which: packer(fields) for which, fields in STRUCTS.items()}


def declare(lib):
    """Prototypes of this module's entry points (called when the library is loaded)."""
    size = ctypes.POINTER(ctypes.c_size_t)
    for name in ("ssm_gated_norm", "ssm_block_norm"):
        for end, last in (("_fwd", _vp), ("_bwd", _vp), ("_bwd_workspace_size", size)):
            fn = getattr(lib, name + end)
            fn.argtypes, fn.restype = [_vp, last], ctypes.c_int
    check_layouts(lib, STRUCTS, _PACKED)


def _gated(x, z, w):
    """(sizes and input type, addresses and strides of x and z, address of w, w_per_head), checked."""
    import torch

    if x.dim() != 4:
        raise ValueError("x must be (B, L, H, d)")
    shape, dt = x.shape, x.dtype
    B, L, H, d = shape
    xs = H * d if x.is_contiguous() else _head_tokens(x, shape, "x", dt)
    zs = xs if z.is_contiguous() and z.dtype is dt and z.shape == shape and xs == H * d else _head_tokens(z, shape, "z", dt)
    per_head = w is not None and w.dim() == 2
    if w is not None:
        _need(w, (H, d) if per_head else (d,), "w", torch.float32)
    return (B, L, H, d, _b._dtype_code(x)), (x.data_ptr(), z.data_ptr(), xs, zs), _at(w), int(per_head)


def ssm_gated_norm_fwd(x, z, *, w=None, eps=1e-6, gate_first=False, out=None, out_dtype=None, stream=None):
    """Norm of x (B, L, H, d) for each head with the gate silu(z), z as x; returns out.

    w (d,) or (H, d) float32, None for 1. The gate multiplies the normed row, or with
    ``gate_first`` the row before the norm. ``out`` is allocated (float32 unless
    ``out_dtype`` says bfloat16) when not given.
    """
    import torch

    lib = _b.load_library()
    sizes, rows, at_w, per_head = _gated(x, z, w)
    if out is None:
        out = _new(x, out_dtype or torch.float32, stream)
    else:
        _need(out, x.shape, "out", out.dtype)
    d = _one_device(x, z, w, out)
    _call(lib.ssm_gated_norm_fwd, _PACKED[10].pack(*sizes, _b._dtype_code(out), *rows, at_w, out.data_ptr(), 0, 0, 0, 0,
                                                   0, 0, eps, bool(gate_first), per_head, 0), stream, d)
    return out


def ssm_gated_norm_bwd(x, z, dout, *, w=None, eps=1e-6, gate_first=False, grad_dtype=None, want_dw=True,
                       workspace=None, stream=None):
    """Gradients of ssm_gated_norm_fwd for the same inputs and the output's gradient.
    Returns a dict with dx, dz in ``grad_dtype`` (float32 by default) and float32 dw as
    w, (d,) without w (None without ``want_dw``)."""
    import torch

    lib = _b.load_library()
    dt = grad_dtype or torch.float32
    sizes, rows, at_w, per_head = _gated(x, z, w)
    _need(dout, x.shape, "dout", x.dtype)
    d = _one_device(x, z, dout, w, workspace)
    g = dict(dx=_new(x, dt, stream), dz=_new(z, dt, stream), dw=None)
    if want_dw:
        g["dw"] = _sum(w, x.shape[3:], x.device, stream)
    head = (*sizes, _b._dtype_code(g["dx"]), *rows, at_w, 0, dout.data_ptr(), *[_at(t) for t in g.values()])
    tail = (eps, bool(gate_first), per_head, 0)
    pack = _PACKED[10].pack
    workspace, at, n = _space(lib.ssm_gated_norm_bwd_workspace_size, pack(*head, 0, 0, *tail), workspace, x.device,
                              stream)
    _call(lib.ssm_gated_norm_bwd, pack(*head, at, n, *tail), stream, d)
    return g


def _block(y, x, w, post, w_post, gate, res_dtype):
    """(sizes, input type, stream type's code, gate_rows, addresses of the inputs, the stream's type), checked."""
    import torch

    if y.dim() != 3:
        raise ValueError("y must be (B, L, D)")
    f32, shape = torch.float32, y.shape
    B, L, D = shape
    ys = D if y.is_contiguous() else _tokens(y, shape, "y", y.dtype)
    if x is not None:
        if res_dtype is not None and res_dtype != x.dtype:
            raise TypeError("res_dtype %s is not the type of x, %s" % (res_dtype, x.dtype))
        res_dtype = x.dtype
        _need(x, shape, "x", res_dtype)
    elif res_dtype is None:
        res_dtype = f32
    if res_dtype is not f32 and res_dtype is not torch.bfloat16:
        raise TypeError("unsupported dtype %s (float32 or bfloat16)" % res_dtype)
    if w is not None:
        _need(w, (D,), "w", f32)
    if w_post is not None:
        if not post:
            raise ValueError("w_post comes with post")
        _need(w_post, (D,), "w_post", f32)
    rows = gate is not None and gate.dim() == 2
    if gate is not None:
        _need(gate, (B, D) if rows else (D,), "gate", f32)
    code = _b.SSM_F32 if res_dtype is f32 else _b.SSM_BF16
    inputs = (code, int(rows), y.data_ptr(), ys, _at(x), _at(w), _at(w_post), _at(gate))
    return (B, L, D, _b._dtype_code(y)), inputs, res_dtype


def ssm_block_norm_fwd(y, x=None, *, w=None, post=False, w_post=None, gate=None, scale=1.0, eps=1e-6, out=None,
                       x_out=None, out_dtype=None, res_dtype=None, want_x=True, stream=None):
    """A block's output y (B, L, D) joins the residual stream x (B, L, D), and the next
    block's input is normed: x_out = x + scale gate m, out = w norm(x_out), with m = y,
    or w_post norm(y) with ``post``. Returns (out, x_out).

    y float32 or bfloat16; x float32 or bfloat16 whatever y is, None where the stream
    starts (x_out then has ``res_dtype``, float32 by default); w, w_post (D,) and gate
    (D,) or (B, D) float32, None for 1. ``out`` is allocated (float32 unless ``out_dtype``
    says bfloat16) when not given; x_out too, or not written without ``want_x``.
    """
    import torch

    lib = _b.load_library()
    sizes, inputs, res = _block(y, x, w, post, w_post, gate, res_dtype)
    if out is None:
        out = _new(y, out_dtype or torch.float32, stream)
    else:
        _need(out, y.shape, "out", out.dtype)
    if x_out is not None:
        _need(x_out, y.shape, "x_out", res)
    elif want_x:
        x_out = _new(y, res, stream)
    d = _one_device(y, x, w, w_post, gate, out, x_out)
    _call(lib.ssm_block_norm_fwd, _PACKED[11].pack(*sizes, _b._dtype_code(out), *inputs, out.data_ptr(), _at(x_out), 0, 0,
                                                   0, 0, 0, 0, 0, 0, 0, eps, scale, bool(post), 0), stream, d)
    return out, x_out


def ssm_block_norm_bwd(y, x, dout, dx_out=None, *, w=None, post=False, w_post=None, gate=None, scale=1.0, eps=1e-6,
                       grad_dtype=None, want_dw=True, workspace=None, stream=None):
    """Gradients of ssm_block_norm_fwd for the same inputs (x None where the stream
    starts) and the gradients of out and of x_out (None for 0, else in the residual
    stream's type).

    Returns a dict with dy in ``grad_dtype`` (float32 by default), dx as x, and float32
    dw (D,), dw_post (D,), dgate as gate; what belongs to an input or option that is not
    there is None (dw excepted), and the last three without ``want_dw``.
    """
    import torch

    lib = _b.load_library()
    sizes, inputs, res = _block(y, x, w, post, w_post, gate, dx_out.dtype if x is None and dx_out is not None else None)
    _need(dout, y.shape, "dout", y.dtype)
    if dx_out is not None:
        _need(dx_out, y.shape, "dx_out", res)
    d = _one_device(y, x, dout, dx_out, w, w_post, gate, workspace)
    D, dev = sizes[2], y.device

    g = dict(dy=_new(y, grad_dtype or torch.float32, stream), dx=None if x is None else _new(x, res, stream), dw=None,
             dw_post=None, dgate=None)
    if want_dw:
        g["dw"] = _sum(w, (D,), dev, stream)
        if post:
            g["dw_post"] = _sum(w_post, (D,), dev, stream)
        if gate is not None:
            g["dgate"] = _sum(gate, None, dev, stream)
    head = (*sizes, _b._dtype_code(g["dy"]), *inputs, 0, 0, dout.data_ptr(), _at(dx_out), *[_at(t) for t in g.values()])
    tail = (eps, scale, bool(post), 0)
    pack = _PACKED[11].pack
    workspace, at, n = _space(lib.ssm_block_norm_bwd_workspace_size, pack(*head, 0, 0, *tail), workspace, dev, stream)
    _call(lib.ssm_block_norm_bwd, pack(*head, at, n, *tail), stream, d)
    return g

"""ctypes binding of the norms around a block (include/ssm_scan.h).

Argument marshalling only, as in binding.py. A mixer's output, its gate and a block's
output may be slices of one packed tensor: entries are dense inside a token, tokens lie a
fixed stride apart, batch rows follow each other. Everything else is contiguous.

Streams as in binding.py: what a call allocates belongs to the stream that it runs on.
"""
from __future__ import annotations

import ctypes

from . import binding as _b
from .binding_delta import _addr, _need, _out, _workspace
from .binding_delta import _tokens as _head_tokens
from .binding_glr import _call, _one_device, _tokens

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


def declare(lib):
    """Prototypes of this module's entry points (called when the library is loaded)."""
    size = ctypes.POINTER(ctypes.c_size_t)
    for name, struct in (("ssm_gated_norm", GatedNormParams), ("ssm_block_norm", BlockNormParams)):
        for end, last in (("_fwd", _vp), ("_bwd", _vp), ("_bwd_workspace_size", size)):
            fn = getattr(lib, name + end)
            fn.argtypes, fn.restype = [ctypes.POINTER(struct), last], ctypes.c_int
    for which, struct in STRUCTS.items():
        if lib.ssm_abi_struct_size(which) != ctypes.sizeof(struct):
            raise ImportError("libssmscan.so struct layout does not match this binding")


def _gated_params(x, z, w, eps, gate_first):
    import torch

    if x.dim() != 4:
        raise ValueError("x must be (B, L, H, d)")
    B, L, H, d = x.shape
    xs = _head_tokens(x, (B, L, H, d), "x", x.dtype)
    zs = _head_tokens(z, (B, L, H, d), "z", x.dtype)
    per_head = w is not None and w.dim() == 2
    if w is not None:
        _need(w, (H, d) if per_head else (d,), "w", torch.float32)
    p = GatedNormParams(B, L, H, d, _b._dtype_code(x), 0, x.data_ptr(), z.data_ptr(), xs, zs, _addr(w))
    p.eps, p.gate_first, p.w_per_head = eps, int(bool(gate_first)), int(per_head)
    return p


def ssm_gated_norm_fwd(x, z, *, w=None, eps=1e-6, gate_first=False, out=None, out_dtype=None, stream=None):
    """Norm of x (B, L, H, d) for each head with the gate silu(z), z as x; returns out.

    w (d,) or (H, d) float32, None for 1. The gate multiplies the normed row, or with
    ``gate_first`` the row before the norm. ``out`` is allocated (float32 unless
    ``out_dtype`` says bfloat16) when not given.
    """
    import torch

    lib = _b.load_library()
    if out is None:
        out = _out(x, out_dtype or torch.float32, stream)
    p = _gated_params(x, z, w, eps, gate_first)
    _need(out, x.shape, "out", out.dtype)
    _one_device(x, z, w, out)
    p.out_dtype, p.out = _b._dtype_code(out), out.data_ptr()
    _call(lib.ssm_gated_norm_fwd, p, stream, x.device)
    return out


def ssm_gated_norm_bwd(x, z, dout, *, w=None, eps=1e-6, gate_first=False, grad_dtype=None, want_dw=True,
                       workspace=None, stream=None):
    """Gradients of ssm_gated_norm_fwd for the same inputs and the output's gradient.
    Returns a dict with dx, dz in ``grad_dtype`` (float32 by default) and float32 dw as
    w, (d,) without w (None without ``want_dw``)."""
    import torch

    lib = _b.load_library()
    dt = grad_dtype or torch.float32
    p = _gated_params(x, z, w, eps, gate_first)
    _need(dout, x.shape, "dout", x.dtype)
    _one_device(x, z, dout, w, workspace)
    g = dict(dx=_out(x, dt, stream), dz=_out(z, dt, stream), dw=None)
    if want_dw:
        g["dw"] = _b._result(x.shape[3:] if w is None else w.shape, torch.float32, x.device, stream)
    p.out_dtype = _b._dtype_code(g["dx"])
    p.dout, p.dx, p.dz, p.dw = dout.data_ptr(), g["dx"].data_ptr(), g["dz"].data_ptr(), _addr(g["dw"])
    workspace = _workspace(lib.ssm_gated_norm_bwd_workspace_size, p, workspace, x.device, stream)
    _call(lib.ssm_gated_norm_bwd, p, stream, x.device)
    return g


def _block_params(y, x, w, post, w_post, gate, scale, eps, res_dtype):
    import torch

    if y.dim() != 3:
        raise ValueError("y must be (B, L, D)")
    B, L, D = y.shape
    ys = _tokens(y, y.shape, "y", y.dtype)
    if x is not None:
        if res_dtype is not None and res_dtype != x.dtype:
            raise TypeError("res_dtype %s is not the type of x, %s" % (res_dtype, x.dtype))
        _need(x, y.shape, "x", x.dtype)
        res_dtype = x.dtype
    if w_post is not None and not post:
        raise ValueError("w_post comes with post")
    for t, name in ((w, "w"), (w_post, "w_post")):
        if t is not None:
            _need(t, (D,), name, torch.float32)
    rows = gate is not None and gate.dim() == 2
    if gate is not None:
        _need(gate, (B, D) if rows else (D,), "gate", torch.float32)
    res_dtype = res_dtype or torch.float32
    if res_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("unsupported dtype %s (float32 or bfloat16)" % res_dtype)
    p = BlockNormParams(B, L, D, _b._dtype_code(y), 0, _b.SSM_BF16 if res_dtype == torch.bfloat16 else _b.SSM_F32,
                        int(rows), y.data_ptr(), ys, _addr(x), _addr(w), _addr(w_post), _addr(gate))
    p.eps, p.scale, p.post = eps, scale, int(bool(post))
    return p, res_dtype


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
    p, res = _block_params(y, x, w, post, w_post, gate, scale, eps, res_dtype)
    if out is None:
        out = _out(y, out_dtype or torch.float32, stream)
    if x_out is None and want_x:
        x_out = _out(y, res, stream)
    _need(out, y.shape, "out", out.dtype)
    if x_out is not None:
        _need(x_out, y.shape, "x_out", res)
    _one_device(y, x, w, w_post, gate, out, x_out)
    p.out_dtype, p.out, p.x_out = _b._dtype_code(out), out.data_ptr(), _addr(x_out)
    _call(lib.ssm_block_norm_fwd, p, stream, y.device)
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
    p, res = _block_params(y, x, w, post, w_post, gate, scale, eps, dx_out.dtype if x is None and dx_out is not None else None)
    _need(dout, y.shape, "dout", y.dtype)
    if dx_out is not None:
        _need(dx_out, y.shape, "dx_out", res)
    _one_device(y, x, dout, dx_out, w, w_post, gate, workspace)
    D, dev = y.shape[2], y.device

    def new(wanted, shape):
        return _b._result(shape, torch.float32, dev, stream) if wanted else None

    g = dict(dy=_out(y, grad_dtype or torch.float32, stream), dx=None if x is None else _out(x, res, stream),
             dw=new(want_dw, (D,)), dw_post=new(want_dw and post, (D,)),
             dgate=new(want_dw and gate is not None, () if gate is None else gate.shape))
    p.out_dtype = _b._dtype_code(g["dy"])
    p.dout, p.dx_out = dout.data_ptr(), _addr(dx_out)
    for name, t in g.items():
        setattr(p, name, _addr(t))
    workspace = _workspace(lib.ssm_block_norm_bwd_workspace_size, p, workspace, dev, stream)
    _call(lib.ssm_block_norm_bwd, p, stream, dev)
    return g

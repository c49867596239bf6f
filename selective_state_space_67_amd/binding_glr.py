"""ctypes binding of the gated linear recurrence (include/ssm_scan.h).

Argument marshalling only, as in binding.py. Tensors u, dt_raw, in_raw, z may be
slices of one packed projection: channels are dense inside a token, tokens lie a
fixed stride apart, batch rows follow each other. Everything else is contiguous.

Streams as in binding.py: what a call allocates belongs to the stream that it runs on.

A small call's time is mostly this module's, so its parameter structs are packed into
bytes in one go (a ctypes structure of twenty fields takes four times as long), and a
tensor that is as expected is looked at no further.
"""
from __future__ import annotations

import ctypes
import struct

from . import binding as _b
from .binding_delta import _need

_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p

SSM_GLR_SIGMOID = 0
SSM_GLR_SOFTPLUS = 1
SSM_GLR_UNIT = 0
SSM_GLR_REST = 1
SSM_GLR_ONE = 2
_DECAYS = {"sigmoid": SSM_GLR_SIGMOID, "softplus": SSM_GLR_SOFTPLUS}
_MIXES = {"unit": SSM_GLR_UNIT, "rest": SSM_GLR_REST, "one": SSM_GLR_ONE}

_INPUTS = [("u", _vp), ("dt_raw", _vp), ("in_raw", _vp), ("z", _vp), ("u_stride", _i64), ("dt_stride", _i64),
           ("in_stride", _i64), ("z_stride", _i64), ("A", _vp), ("dt_bias", _vp), ("in_bias", _vp)]


class GlrParams(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("dim", _i64), ("in_dtype", _i32), ("out_dtype", _i32)] + _INPUTS + [
        ("reset", _vp), ("h0", _vp), ("out", _vp), ("h_last", _vp), ("dout", _vp), ("dh_last", _vp), ("du", _vp),
        ("d_dt_raw", _vp), ("din_raw", _vp), ("dz", _vp), ("dA", _vp), ("d_dt_bias", _vp), ("din_bias", _vp),
        ("dh0", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("decay", _i32), ("mix", _i32)]


class GlrUpdateParams(ctypes.Structure):
    _fields_ = [("batch", _i64), ("tokens", _i64), ("dim", _i64), ("in_dtype", _i32), ("out_dtype", _i32),
                ("h", _vp)] + _INPUTS + [("out", _vp), ("decay", _i32), ("mix", _i32)]


STRUCTS = {8: GlrParams, 9: GlrUpdateParams}
_CODES = {_i64: "q", _i32: "i", _vp: "Q", ctypes.c_size_t: "Q", ctypes.c_float: "f"}


def packer(fields):
    """Packs a parameter struct's fields, in order and at the places that C gives them."""
    return struct.Struct("@" + "".join(_CODES[t] for _, t in fields._fields_))


_PACKED = {which: packer(fields) for which, fields in STRUCTS.items()}


def declare(lib):
    """Prototypes of this module's entry points (called when the library is loaded). A
    parameter struct is passed by reference or as packed bytes."""
    size = ctypes.POINTER(ctypes.c_size_t)
    for name, last in (("ssm_glr_fwd", _vp), ("ssm_glr_bwd", _vp), ("ssm_glr_update", _vp),
                       ("ssm_glr_workspace_size", size), ("ssm_glr_bwd_workspace_size", size)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [_vp, last], ctypes.c_int
    check_layouts(lib, STRUCTS, _PACKED)


def check_layouts(lib, structs, packed):
    for which, fields in structs.items():
        if not lib.ssm_abi_struct_size(which) == ctypes.sizeof(fields) == packed[which].size:
            raise ImportError("libssmscan.so struct layout does not match this binding")


def _one_device(first, *others):
    """Everything lies where the call runs (an address on another device would fault there): its number."""
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("tensors on %s and %s in one call" % (first.device, t.device))
    return d


def _call(fn, packed, stream, device):
    """Enqueue on the stream, with its device (a number) current."""
    import torch

    c = torch._C
    if device < 0:
        if isinstance(fn, ctypes._CFuncPtr):  # (a stand-in may have them anywhere)
            raise ValueError("tensors on cpu: the operators run on a GPU")
        status = fn(packed, 0 if stream is None else stream.cuda_stream)
    else:
        st = c._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
        if device == c._cuda_getDevice():
            status = fn(packed, st)
        else:
            with torch.cuda.device(device):
                status = fn(packed, st)
    if status != 0:
        _b._check(status)


def _at(t):
    return 0 if t is None else t.data_ptr()


def _new(t, dtype, stream):
    """A contiguous output of t's shape."""
    import torch

    if stream is None:
        if t.dtype is dtype and t.is_contiguous():
            return torch.empty_like(t)
        return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)
    return _b._result(t.shape, dtype, t.device, stream)


def _sum(like, shape, device, stream):
    """A float32 output of this shape, which `like` has if there is one."""
    import torch

    if like is not None:
        return _new(like, torch.float32, stream)
    return _b._result(shape, torch.float32, device, stream)


def _space(size_fn, packed, workspace, device, stream):
    """(workspace, its address and bytes) of what a call needs."""
    import torch

    n = ctypes.c_size_t(0)
    _b._check(size_fn(packed, ctypes.byref(n)))
    if n.value == 0:
        return workspace, 0, 0
    if workspace is None or workspace.numel() * workspace.element_size() < n.value or not workspace.is_contiguous():
        workspace = _b._empty(int(n.value), torch.uint8, device, stream)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _tokens(t, shape, name, dtype):
    """Elements between consecutive tokens of t (B, L, D)."""
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    B, L, D = shape
    if t.is_contiguous() or t.numel() == 0:
        return D
    s = t.stride()
    step = s[1] if L > 1 else s[0] if B > 1 else D
    if (D > 1 and s[2] != 1) or (L > 1 and B > 1 and s[0] != L * step) or step < D:
        raise ValueError("%s must have dense channels inside a token and tokens a fixed stride apart" % name)
    return step


def _inputs(u, dt_raw, A, dt_bias, in_raw, in_bias, z, decay, mix):
    """(sizes and input type, the struct fields _INPUTS, the kinds), checked."""
    import torch

    f32 = torch.float32
    p_decay, p_mix = _DECAYS.get(decay), _MIXES.get(mix)
    if p_decay is None:
        raise ValueError("decay is 'sigmoid' or 'softplus' (got %r)" % (decay,))
    if p_mix is None:
        raise ValueError("mix is 'unit', 'rest' or 'one' (got %r)" % (mix,))
    if u.dim() != 3:
        raise ValueError("u must be (B, L, D)")
    shape, dt = u.shape, u.dtype
    B, L, D = shape
    us = D if u.is_contiguous() else _tokens(u, shape, "u", dt)
    ds = D if dt_raw.is_contiguous() and dt_raw.dtype is dt and dt_raw.shape == shape else _tokens(dt_raw, shape, "dt_raw", dt)
    ins = zs = at_in = at_z = at_dt_bias = at_in_bias = 0
    if in_raw is not None:
        ins = D if in_raw.is_contiguous() and in_raw.dtype is dt and in_raw.shape == shape else _tokens(in_raw, shape, "in_raw", dt)
        at_in = in_raw.data_ptr()
    elif in_bias is not None:
        raise ValueError("in_bias comes with in_raw")
    if z is not None:
        zs = D if z.is_contiguous() and z.dtype is dt and z.shape == shape else _tokens(z, shape, "z", dt)
        at_z = z.data_ptr()
    size = (D,)
    _need(A, size, "A", f32)
    if dt_bias is not None:
        _need(dt_bias, size, "dt_bias", f32)
        at_dt_bias = dt_bias.data_ptr()
    if in_bias is not None:
        _need(in_bias, size, "in_bias", f32)
        at_in_bias = in_bias.data_ptr()
    fields = (u.data_ptr(), dt_raw.data_ptr(), at_in, at_z, us, ds, ins, zs, A.data_ptr(), at_dt_bias, at_in_bias)
    return (B, L, D, _b._dtype_code(u)), fields, (p_decay, p_mix)


def _sequence(sizes, reset, h0):
    """Addresses of reset and h0, checked."""
    import torch

    B, L, D, _ = sizes
    if reset is not None:
        _need(reset, (B, L), "reset", torch.uint8)
    if h0 is not None:
        _need(h0, (B, D), "h0", torch.float32)
    return _at(reset), _at(h0)


_NO_GRADS = (0,) * 10


def ssm_glr_fwd(u, dt_raw, A, *, dt_bias=None, in_raw=None, in_bias=None, z=None, reset=None, h0=None, out=None,
                h_last=None, out_dtype=None, decay="sigmoid", mix="unit", workspace=None, stream=None):
    """Gated linear recurrence over the whole sequence; returns ``out`` (B, L, D).

    u, dt_raw, in_raw, z: (B, L, D) float32 or bfloat16 (the last two optional); A,
    dt_bias, in_bias: (D,) float32; reset: (B, L) uint8; h0, h_last: (B, D) float32.
    ``decay`` "sigmoid" or "softplus", ``mix`` "unit", "rest" or "one" (see
    include/ssm_scan.h). ``out`` is allocated (float32 unless ``out_dtype`` says
    bfloat16) when not given, and so is the workspace the library asks for.
    """
    import torch

    lib = _b.load_library()
    sizes, fields, kinds = _inputs(u, dt_raw, A, dt_bias, in_raw, in_bias, z, decay, mix)
    if out is None:
        out = _new(u, out_dtype or torch.float32, stream)
    else:
        _need(out, u.shape, "out", out.dtype)
    if h_last is not None:
        _need(h_last, (sizes[0], sizes[2]), "h_last", torch.float32)
    d = _one_device(u, dt_raw, A, dt_bias, in_raw, in_bias, z, reset, h0, out, h_last, workspace)
    head = (*sizes, _b._dtype_code(out), *fields, *_sequence(sizes, reset, h0), out.data_ptr(), _at(h_last), *_NO_GRADS)
    pack = _PACKED[8].pack
    workspace, at, n = _space(lib.ssm_glr_workspace_size, pack(*head, 0, 0, *kinds), workspace,
                              u.device, stream)
    _call(lib.ssm_glr_fwd, pack(*head, at, n, *kinds), stream, d)
    return out


def _update(h, u, dt_raw, A, dt_bias, in_raw, in_bias, z, out, out_dtype, decay, mix, stream):
    """(packed struct, out, device) of a decode window."""
    import torch

    sizes, fields, kinds = _inputs(u, dt_raw, A, dt_bias, in_raw, in_bias, z, decay, mix)
    if out is None:
        out = _new(u, out_dtype or torch.float32, stream)
    else:
        _need(out, u.shape, "out", out.dtype)
    _need(h, (sizes[0], sizes[2]), "h", torch.float32)
    d = _one_device(u, h, dt_raw, A, dt_bias, in_raw, in_bias, z, out)
    return _PACKED[9].pack(*sizes, _b._dtype_code(out), h.data_ptr(), *fields, out.data_ptr(), *kinds), out, d


def ssm_glr_update(h, u, dt_raw, A, *, dt_bias=None, in_raw=None, in_bias=None, z=None, out=None, out_dtype=None,
                   decay="sigmoid", mix="unit", stream=None):
    """Decode window of T tokens: updates h (B, D) float32 in place and returns out
    (B, T, D). Arguments as for ssm_glr_fwd with L = T."""
    lib = _b.load_library()
    packed, out, d = _update(h, u, dt_raw, A, dt_bias, in_raw, in_bias, z, out, out_dtype, decay, mix, stream)
    _call(lib.ssm_glr_update, packed, stream, d)
    return out


def prepare_glr_update(h, u, dt_raw, A, *, dt_bias=None, in_raw=None, in_bias=None, z=None, out=None, out_dtype=None,
                       decay="sigmoid", mix="unit", stream=None):
    """Marshal the arguments of ssm_glr_update once; returns a no-argument callable
    that enqueues the same window again on the same stream (updating h every time)."""
    import torch

    lib = _b.load_library()
    packed, out, d = _update(h, u, dt_raw, A, dt_bias, in_raw, in_bias, z, out, out_dtype, decay, mix, stream)
    fn = lib.ssm_glr_update
    if stream is None and d >= 0:
        stream = torch.cuda.current_stream(d)

    def call():
        _call(fn, packed, stream, d)
        return out

    call.keep = (h, u, dt_raw, A, dt_bias, in_raw, in_bias, z, out)
    return call


def ssm_glr_bwd(u, dt_raw, A, dout, *, dt_bias=None, in_raw=None, in_bias=None, z=None, reset=None, h0=None,
                dh_last=None, grad_dtype=None, decay="sigmoid", mix="unit", want_dh0=True, workspace=None, stream=None):
    """Backward pass of ssm_glr_fwd for the same inputs and the output gradient dout
    (B, L, D).

    Returns a dict with du, d_dt_raw, din_raw, dz in ``grad_dtype`` (float32 by
    default) and float32 dA, d_dt_bias, din_bias (D,), dh0 (B, D); what belongs to an
    input that is not there is None (d_dt_bias excepted), and dh0 when not asked for.
    dh_last is the gradient reaching h_last (None = 0). The workspace is allocated when
    not given or too small.
    """
    import torch

    lib = _b.load_library()
    sizes, fields, kinds = _inputs(u, dt_raw, A, dt_bias, in_raw, in_bias, z, decay, mix)
    gd, f32, dev = grad_dtype or torch.float32, torch.float32, u.device
    B, L, D, _ = sizes
    _need(dout, u.shape, "dout", u.dtype)
    if dh_last is not None:
        _need(dh_last, (B, D), "dh_last", f32)
    d = _one_device(u, dt_raw, A, dout, dt_bias, in_raw, in_bias, z, reset, h0, dh_last, workspace)
    gate = in_raw is not None
    g = dict(du=_new(u, gd, stream), d_dt_raw=_new(u, gd, stream), din_raw=_new(u, gd, stream) if gate else None,
             dz=None if z is None else _new(u, gd, stream), dA=_new(A, f32, stream), d_dt_bias=_new(A, f32, stream),
             din_bias=_new(A, f32, stream) if gate else None, dh0=None)
    if want_dh0:
        g["dh0"] = _sum(h0 if dh_last is None else dh_last, (B, D), dev, stream)
    head = (*sizes, _b._dtype_code(g["du"]), *fields, *_sequence(sizes, reset, h0), 0, 0, dout.data_ptr(), _at(dh_last),
            *[_at(t) for t in g.values()])
    pack = _PACKED[8].pack
    workspace, at, n = _space(lib.ssm_glr_bwd_workspace_size, pack(*head, 0, 0, *kinds), workspace, dev, stream)
    _call(lib.ssm_glr_bwd, pack(*head, at, n, *kinds), stream, d)
    return g

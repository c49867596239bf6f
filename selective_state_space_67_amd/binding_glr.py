"""ctypes binding of the gated linear recurrence (include/ssm_scan.h).

Argument marshalling only, as in binding.py. Tensors u, dt_raw, in_raw, z may be
slices of one packed projection: channels are dense inside a token, tokens lie a
fixed stride apart, batch rows follow each other. Everything else is contiguous.

Streams as in binding.py: what a call allocates belongs to the stream that it runs on.
"""
from __future__ import annotations

import ctypes

from . import binding as _b
from .binding_delta import _addr, _need, _out, _stream, _workspace

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
        ("dh0", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("decay", _i32), ("mix", _i32),
        ("num_segments", _i32), ("reserved0", _i32)]


class GlrUpdateParams(ctypes.Structure):
    _fields_ = [("batch", _i64), ("tokens", _i64), ("dim", _i64), ("in_dtype", _i32), ("out_dtype", _i32),
                ("h", _vp)] + _INPUTS + [("out", _vp), ("decay", _i32), ("mix", _i32)]


STRUCTS = {8: GlrParams, 9: GlrUpdateParams}


def declare(lib):
    """Prototypes of this module's entry points (called when the library is loaded)."""
    size = ctypes.POINTER(ctypes.c_size_t)
    for name, struct in (("ssm_glr_fwd", GlrParams), ("ssm_glr_bwd", GlrParams), ("ssm_glr_update", GlrUpdateParams)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [ctypes.POINTER(struct), _vp], ctypes.c_int
    for name in ("ssm_glr_workspace_size", "ssm_glr_bwd_workspace_size"):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [ctypes.POINTER(GlrParams), size], ctypes.c_int
    for which, struct in STRUCTS.items():
        if lib.ssm_abi_struct_size(which) != ctypes.sizeof(struct):
            raise ImportError("libssmscan.so struct layout does not match this binding")


def _one_device(first, *others):
    """Everything lies where the call runs (an address on another device would fault there)."""
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError("tensors on %s and %s in one call" % (first.device, t.device))


def _call(fn, p, stream, device):
    """Enqueue on the stream, with its device current."""
    import torch

    st = _stream(stream, device)
    if device.type != "cuda" or device.index == torch._C._cuda_getDevice():
        _b._check(fn(ctypes.byref(p), st))
        return
    with torch.cuda.device(device):
        _b._check(fn(ctypes.byref(p), st))


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
    """The struct fields _INPUTS and the kinds, checked."""
    import torch

    if decay not in _DECAYS:
        raise ValueError("decay is 'sigmoid' or 'softplus' (got %r)" % (decay,))
    if mix not in _MIXES:
        raise ValueError("mix is 'unit', 'rest' or 'one' (got %r)" % (mix,))
    if in_bias is not None and in_raw is None:
        raise ValueError("in_bias comes with in_raw")
    if u.dim() != 3:
        raise ValueError("u must be (B, L, D)")
    shape, dt = u.shape, u.dtype
    D = shape[2]
    steps = [_tokens(u, shape, "u", dt), _tokens(dt_raw, shape, "dt_raw", dt),
             0 if in_raw is None else _tokens(in_raw, shape, "in_raw", dt),
             0 if z is None else _tokens(z, shape, "z", dt)]
    _need(A, (D,), "A", torch.float32)
    if dt_bias is not None:
        _need(dt_bias, (D,), "dt_bias", torch.float32)
    if in_bias is not None:
        _need(in_bias, (D,), "in_bias", torch.float32)
    fields = (u.data_ptr(), dt_raw.data_ptr(), _addr(in_raw), _addr(z), *steps, A.data_ptr(), _addr(dt_bias),
              _addr(in_bias))
    return fields, _DECAYS[decay], _MIXES[mix]


def _params(u, fields, reset, h0, out_code):
    import torch

    B, L, D = u.shape
    if reset is not None:
        _need(reset, (B, L), "reset", torch.uint8)
    if h0 is not None:
        _need(h0, (B, D), "h0", torch.float32)
    return GlrParams(B, L, D, _b._dtype_code(u), out_code, *fields, _addr(reset), _addr(h0))


def ssm_glr_fwd(u, dt_raw, A, *, dt_bias=None, in_raw=None, in_bias=None, z=None, reset=None, h0=None, out=None,
                h_last=None, out_dtype=None, decay="sigmoid", mix="unit", num_segments=0, workspace=None, stream=None):
    """Gated linear recurrence over the whole sequence; returns ``out`` (B, L, D).

    u, dt_raw, in_raw, z: (B, L, D) float32 or bfloat16 (the last two optional); A,
    dt_bias, in_bias: (D,) float32; reset: (B, L) uint8; h0, h_last: (B, D) float32.
    ``decay`` "sigmoid" or "softplus", ``mix`` "unit", "rest" or "one" (see
    include/ssm_scan.h). ``out`` is allocated (float32 unless ``out_dtype`` says
    bfloat16) when not given, and so is the workspace the library asks for.
    """
    import torch

    lib = _b.load_library()
    fields, p_decay, p_mix = _inputs(u, dt_raw, A, dt_bias, in_raw, in_bias, z, decay, mix)
    if out is None:
        out = _out(u, out_dtype or torch.float32, stream)
    _need(out, u.shape, "out", out.dtype)
    p = _params(u, fields, reset, h0, _b._dtype_code(out))
    if h_last is not None:
        _need(h_last, (p.batch, p.dim), "h_last", torch.float32)
    p.out, p.h_last = out.data_ptr(), _addr(h_last)
    p.decay, p.mix, p.num_segments = p_decay, p_mix, num_segments
    workspace = _workspace(lib.ssm_glr_workspace_size, p, workspace, u.device, stream)
    _one_device(u, dt_raw, A, dt_bias, in_raw, in_bias, z, reset, h0, out, h_last, workspace)
    _call(lib.ssm_glr_fwd, p, stream, u.device)
    return out


def _update_params(h, u, dt_raw, A, dt_bias, in_raw, in_bias, z, out, decay, mix):
    import torch

    fields, p_decay, p_mix = _inputs(u, dt_raw, A, dt_bias, in_raw, in_bias, z, decay, mix)
    B, T, D = u.shape
    _need(h, (B, D), "h", torch.float32)
    _need(out, u.shape, "out", out.dtype)
    _one_device(u, h, dt_raw, A, dt_bias, in_raw, in_bias, z, out)
    return GlrUpdateParams(B, T, D, _b._dtype_code(u), _b._dtype_code(out), h.data_ptr(), *fields, out.data_ptr(),
                           p_decay, p_mix)


def ssm_glr_update(h, u, dt_raw, A, *, dt_bias=None, in_raw=None, in_bias=None, z=None, out=None, out_dtype=None,
                   decay="sigmoid", mix="unit", stream=None):
    """Decode window of T tokens: updates h (B, D) float32 in place and returns out
    (B, T, D). Arguments as for ssm_glr_fwd with L = T."""
    import torch

    lib = _b.load_library()
    if out is None:
        out = _out(u, out_dtype or torch.float32, stream)
    p = _update_params(h, u, dt_raw, A, dt_bias, in_raw, in_bias, z, out, decay, mix)
    _call(lib.ssm_glr_update, p, stream, u.device)
    return out


def prepare_glr_update(h, u, dt_raw, A, *, dt_bias=None, in_raw=None, in_bias=None, z=None, out=None, out_dtype=None,
                       decay="sigmoid", mix="unit", stream=None):
    """Marshal the arguments of ssm_glr_update once; returns a no-argument callable
    that enqueues the same window again (updating h every time)."""
    import torch

    lib = _b.load_library()
    if out is None:
        out = _out(u, out_dtype or torch.float32, stream)
    p = _update_params(h, u, dt_raw, A, dt_bias, in_raw, in_bias, z, out, decay, mix)
    fn, dev = lib.ssm_glr_update, u.device
    if stream is None and dev.type == "cuda":
        stream = torch.cuda.current_stream(dev)

    def call():
        _call(fn, p, stream, dev)
        return out

    call.keep = ((h, u, dt_raw, A, dt_bias, in_raw, in_bias, z, out), p)
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
    fields, p_decay, p_mix = _inputs(u, dt_raw, A, dt_bias, in_raw, in_bias, z, decay, mix)
    gd, f32, dev = grad_dtype or torch.float32, torch.float32, u.device
    B, L, D = u.shape
    _need(dout, u.shape, "dout", u.dtype)
    if dh_last is not None:
        _need(dh_last, (B, D), "dh_last", f32)

    def new(wanted, shape, dtype):
        return _b._result(shape, dtype, dev, stream) if wanted else None

    gate = in_raw is not None
    g = dict(du=new(True, u.shape, gd), d_dt_raw=new(True, u.shape, gd), din_raw=new(gate, u.shape, gd),
             dz=new(z is not None, u.shape, gd), dA=new(True, (D,), f32), d_dt_bias=new(True, (D,), f32),
             din_bias=new(gate, (D,), f32), dh0=new(want_dh0, (B, D), f32))
    p = _params(u, fields, reset, h0, _b._dtype_code(g["du"]))
    p.dout, p.dh_last = dout.data_ptr(), _addr(dh_last)
    for name, t in g.items():
        setattr(p, name, _addr(t))
    p.decay, p.mix = p_decay, p_mix
    workspace = _workspace(lib.ssm_glr_bwd_workspace_size, p, workspace, dev, stream)
    _one_device(u, dt_raw, A, dout, dt_bias, in_raw, in_bias, z, reset, h0, dh_last, workspace)
    _call(lib.ssm_glr_bwd, p, stream, dev)
    return g

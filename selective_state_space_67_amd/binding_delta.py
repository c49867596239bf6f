"""ctypes binding of the gated delta rule and of the head norms (include/ssm_scan.h).

Argument marshalling only, as in binding.py. Tensors q, k, v may be slices of
one packed projection: heads are dense inside a token, tokens lie a fixed
stride apart, batch rows follow each other. Everything else is contiguous.

Streams as in binding.py: what a call allocates belongs to the stream that it runs on.
"""
from __future__ import annotations

import ctypes

from . import binding as _b

_i64, _i32, _vp, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float

SSM_NORM_RMS = 0
SSM_NORM_L2 = 1
_NORM_KINDS = {"rms": SSM_NORM_RMS, "l2": SSM_NORM_L2}

_HEAD = [("batch", _i64), ("seqlen", _i64), ("key_heads", _i64), ("value_heads", _i64), ("dk", _i64), ("dv", _i64),
         ("in_dtype", _i32)]
_QKV = [("q", _vp), ("k", _vp), ("v", _vp), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
        ("dt_raw", _vp), ("beta_raw", _vp), ("dt_bias", _vp), ("A", _vp)]


class DeltaParams(ctypes.Structure):
    _fields_ = _HEAD + [("out_dtype", _i32)] + _QKV + [
        ("reset", _vp), ("h0", _vp), ("out", _vp), ("h_last", _vp), ("workspace", _vp),
        ("workspace_bytes", ctypes.c_size_t), ("scale", _f32), ("beta_scale", _f32), ("num_segments", _i32),
        ("reserved0", _i32)]


class DeltaUpdateParams(ctypes.Structure):
    _fields_ = [("batch", _i64), ("tokens", _i64)] + _HEAD[2:] + [("out_dtype", _i32), ("h", _vp)] + _QKV + [
        ("out", _vp), ("scale", _f32), ("beta_scale", _f32)]


class DeltaBwdParams(ctypes.Structure):
    _fields_ = _HEAD + [("grad_dtype", _i32)] + _QKV + [
        ("reset", _vp), ("h0", _vp), ("dout", _vp), ("dh_last", _vp), ("dq", _vp), ("dk_out", _vp), ("dv_out", _vp),
        ("d_dt_raw", _vp), ("dbeta_raw", _vp), ("dA", _vp), ("d_dt_bias", _vp), ("dh0", _vp), ("workspace", _vp),
        ("workspace_bytes", ctypes.c_size_t), ("scale", _f32), ("beta_scale", _f32)]


class QkNormParams(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("q_heads", _i64), ("k_heads", _i64), ("head_dim", _i64),
                ("rot_dim", _i64), ("rot_positions", _i64), ("in_dtype", _i32), ("out_dtype", _i32),
                ("q", _vp), ("k", _vp), ("q_stride", _i64), ("k_stride", _i64), ("wq", _vp), ("wk", _vp),
                ("cos", _vp), ("sin", _vp), ("positions", _vp), ("q_out", _vp), ("k_out", _vp), ("dq_out", _vp),
                ("dk_out", _vp), ("dq", _vp), ("dk", _vp), ("dwq", _vp), ("dwk", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("eps", _f32), ("norm_kind", _i32), ("interleaved", _i32),
                ("reserved0", _i32)]


STRUCTS = {3: DeltaParams, 4: DeltaUpdateParams, 5: DeltaBwdParams, 6: QkNormParams}


def declare(lib):
    """Prototypes of this module's entry points (called when the library is loaded)."""
    size = ctypes.POINTER(ctypes.c_size_t)
    for name, struct in (("ssm_delta_fwd", DeltaParams), ("ssm_delta_update", DeltaUpdateParams),
                         ("ssm_delta_bwd", DeltaBwdParams),
                         ("ssm_qk_norm_fwd", QkNormParams), ("ssm_qk_norm_bwd", QkNormParams)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [ctypes.POINTER(struct), _vp], ctypes.c_int
    for name, struct in (("ssm_delta_workspace_size", DeltaParams),
                         ("ssm_delta_bwd_workspace_size", DeltaBwdParams),
                         ("ssm_qk_norm_bwd_workspace_size", QkNormParams)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [ctypes.POINTER(struct), size], ctypes.c_int
    for which, struct in STRUCTS.items():
        if lib.ssm_abi_struct_size(which) != ctypes.sizeof(struct):
            raise ImportError("libssmscan.so struct layout does not match this binding")


def _need(t, shape, name, dtype):
    """t is a contiguous tensor of this shape and type (these checks are most of a small call's time)."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        _b._need(t, shape, name, dtype)


def _stream(stream, device):
    """The stream's address; without one, torch's current stream of the device."""
    if stream is not None:
        return stream.cuda_stream
    import torch

    return torch._C._cuda_getCurrentRawStream(device.index)


def _addr(t):
    return None if t is None else t.data_ptr()


def _tokens(t, shape, name, dtype):
    """Elements between consecutive tokens of t (B, L, heads, entries); 0 where there is at most one."""
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    if t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    B, L, H, d = shape
    size = H * d
    if t.is_contiguous() or t.numel() == 0:
        return size
    s = t.stride()
    step = s[1] if L > 1 else s[0]
    if (d > 1 and s[3] != 1) or (H > 1 and s[2] != d) or (L > 1 and B > 1 and s[0] != L * step) or step < size:
        raise ValueError("%s must have dense heads inside a token and tokens a fixed stride apart" % name)
    return step


def _out(t, dtype, stream):
    """An output of t's shape (torch's empty_like would keep t's strides)."""
    import torch

    if stream is None:
        return torch.empty(t.shape, dtype=dtype, device=t.device)
    return _b._result(t.shape, dtype, t.device, stream)


def _workspace(size_fn, p, workspace, device, stream):
    import torch

    n = ctypes.c_size_t(0)
    _b._check(size_fn(ctypes.byref(p), ctypes.byref(n)))
    if n.value:
        if workspace is None or workspace.numel() * workspace.element_size() < n.value:
            workspace = _b._empty(int(n.value), torch.uint8, device, stream)
        p.workspace = workspace.data_ptr()
        p.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def _delta_inputs(q, k, v, dt_raw, A, beta_raw, dt_bias):
    """Sizes and token strides of the delta rule's inputs, checked."""
    import torch

    B, L, Hk, dk = q.shape
    Hv, dv = v.shape[2:]
    qs = _tokens(q, (B, L, Hk, dk), "q", q.dtype)
    ks = _tokens(k, (B, L, Hk, dk), "k", q.dtype)
    vs = _tokens(v, (B, L, Hv, dv), "v", q.dtype)
    _need(dt_raw, (B, L, Hv), "dt_raw", q.dtype)
    _need(beta_raw, (B, L, Hv), "beta_raw", q.dtype)
    _need(A, (Hv,), "A", torch.float32)
    if dt_bias is not None:
        _need(dt_bias, (Hv,), "dt_bias", torch.float32)
    return (B, L, Hk, Hv, dk, dv), (qs, ks, vs)


def _delta_params(q, k, v, dt_raw, A, beta_raw, dt_bias, reset, h0, h_last, out, scale, beta_scale, num_segments):
    import torch

    sizes, strides = _delta_inputs(q, k, v, dt_raw, A, beta_raw, dt_bias)
    B, L, _, Hv, dk, dv = sizes
    _need(out, (B, L, Hv, dv), "out", out.dtype)
    if reset is not None:
        _need(reset, (B, L), "reset", torch.uint8)
    for t, name in ((h0, "h0"), (h_last, "h_last")):
        if t is not None:
            _need(t, (B, Hv, dk, dv), name, torch.float32)
    return DeltaParams(*sizes, _b._dtype_code(q), _b._dtype_code(out), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                       *strides, dt_raw.data_ptr(), beta_raw.data_ptr(), _addr(dt_bias), A.data_ptr(), _addr(reset),
                       _addr(h0), out.data_ptr(), _addr(h_last), None, 0,
                       dk ** -0.5 if scale is None else scale, beta_scale, num_segments, 0)


def ssm_delta_fwd(q, k, v, dt_raw, A, beta_raw, *, dt_bias=None, reset=None, h0=None, out=None, h_last=None,
                  out_dtype=None, scale=None, beta_scale=1.0, num_segments=0, workspace=None, stream=None):
    """Gated delta rule over the whole sequence; returns ``out`` (B, L, Hv, dv).

    q, k: (B, L, Hk, dk), v: (B, L, Hv, dv) with Hv a multiple of Hk, dt_raw and
    beta_raw: (B, L, Hv), all float32 or bfloat16; A, dt_bias: (Hv,) float32;
    reset: (B, L) uint8; h0, h_last: (B, Hv, dk, dv) float32. ``scale`` is
    dk ** -0.5 unless given. ``out`` is allocated (float32 unless ``out_dtype``
    says bfloat16) when not given, and so is the workspace the library asks for.
    """
    import torch

    lib = _b.load_library()
    if out is None:
        out = _out(v, out_dtype or torch.float32, stream)
    p = _delta_params(q, k, v, dt_raw, A, beta_raw, dt_bias, reset, h0, h_last, out, scale, beta_scale, num_segments)
    workspace = _workspace(lib.ssm_delta_workspace_size, p, workspace, v.device, stream)
    _b._check(lib.ssm_delta_fwd(ctypes.byref(p), _stream(stream, v.device)))
    return out


def _delta_update_params(h, q, k, v, dt_raw, A, beta_raw, dt_bias, out, scale, beta_scale):
    import torch

    sizes, strides = _delta_inputs(q, k, v, dt_raw, A, beta_raw, dt_bias)
    B, T, _, Hv, dk, dv = sizes
    _need(h, (B, Hv, dk, dv), "h", torch.float32)
    _need(out, (B, T, Hv, dv), "out", out.dtype)
    return DeltaUpdateParams(*sizes, _b._dtype_code(q), _b._dtype_code(out), h.data_ptr(), q.data_ptr(), k.data_ptr(),
                             v.data_ptr(), *strides, dt_raw.data_ptr(), beta_raw.data_ptr(), _addr(dt_bias),
                             A.data_ptr(), out.data_ptr(), dk ** -0.5 if scale is None else scale, beta_scale)


def ssm_delta_update(h, q, k, v, dt_raw, A, beta_raw, *, dt_bias=None, out=None, out_dtype=None, scale=None,
                     beta_scale=1.0, stream=None):
    """Decode window of T tokens: updates h (B, Hv, dk, dv) float32 in place and
    returns out (B, T, Hv, dv). Arguments as for ssm_delta_fwd with L = T."""
    import torch

    lib = _b.load_library()
    if out is None:
        out = _out(v, out_dtype or torch.float32, stream)
    p = _delta_update_params(h, q, k, v, dt_raw, A, beta_raw, dt_bias, out, scale, beta_scale)
    _b._check(lib.ssm_delta_update(ctypes.byref(p), _stream(stream, v.device)))
    return out


def prepare_delta_update(h, q, k, v, dt_raw, A, beta_raw, *, dt_bias=None, out=None, out_dtype=None, scale=None,
                         beta_scale=1.0, stream=None):
    """Marshal the arguments of ssm_delta_update once; returns a no-argument
    callable that enqueues the same window again (updating h every time)."""
    import torch

    lib = _b.load_library()
    if out is None:
        out = _out(v, out_dtype or torch.float32, stream)
    p = _delta_update_params(h, q, k, v, dt_raw, A, beta_raw, dt_bias, out, scale, beta_scale)
    st, fn, pref = _stream(stream, v.device), lib.ssm_delta_update, ctypes.byref(p)

    def call():
        _b._check(fn(pref, st))
        return out

    call.keep = ((h, q, k, v, dt_raw, A, beta_raw, dt_bias, out), p)
    return call


def ssm_delta_bwd(q, k, v, dt_raw, A, beta_raw, dout, *, dt_bias=None, reset=None, h0=None, dh_last=None,
                  grad_dtype=None, scale=None, beta_scale=1.0, want_d_dt_bias=True, want_dh0=True, workspace=None,
                  stream=None):
    """Backward pass of ssm_delta_fwd for the same inputs and the output gradient
    dout (B, L, Hv, dv).

    Returns a dict with dq, dk, dv, d_dt_raw, dbeta_raw in ``grad_dtype`` (float32 by
    default) and float32 dA, d_dt_bias (Hv,), dh0 (B, Hv, dk, dv) (the last two None
    when not asked for). dh_last is the gradient reaching h_last (None = 0). The
    workspace is allocated when not given or too small.
    """
    import torch

    lib = _b.load_library()
    sizes, strides = _delta_inputs(q, k, v, dt_raw, A, beta_raw, dt_bias)
    B, L, Hk, Hv, dk, dv = sizes
    _need(dout, (B, L, Hv, dv), "dout", q.dtype)
    if reset is not None:
        _need(reset, (B, L), "reset", torch.uint8)
    for t, name in ((h0, "h0"), (dh_last, "dh_last")):
        if t is not None:
            _need(t, (B, Hv, dk, dv), name, torch.float32)
    gd, f32, dev = grad_dtype or torch.float32, torch.float32, q.device

    def new(shape, dtype):
        return _b._result(shape, dtype, dev, stream)

    g = dict(dq=new((B, L, Hk, dk), gd), dk=new((B, L, Hk, dk), gd), dv=new((B, L, Hv, dv), gd),
             d_dt_raw=new((B, L, Hv), gd), dbeta_raw=new((B, L, Hv), gd), dA=new((Hv,), f32),
             d_dt_bias=new((Hv,), f32) if want_d_dt_bias else None, dh0=new((B, Hv, dk, dv), f32) if want_dh0 else None)
    p = DeltaBwdParams(*sizes, _b._dtype_code(q), _b._dtype_code(g["dq"]), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                       *strides, dt_raw.data_ptr(), beta_raw.data_ptr(), _addr(dt_bias), A.data_ptr(), _addr(reset),
                       _addr(h0), dout.data_ptr(), _addr(dh_last), g["dq"].data_ptr(), g["dk"].data_ptr(),
                       g["dv"].data_ptr(), g["d_dt_raw"].data_ptr(), g["dbeta_raw"].data_ptr(), g["dA"].data_ptr(),
                       _addr(g["d_dt_bias"]), _addr(g["dh0"]), None, 0, dk ** -0.5 if scale is None else scale, beta_scale)
    workspace = _workspace(lib.ssm_delta_bwd_workspace_size, p, workspace, dev, stream)
    _b._check(lib.ssm_delta_bwd(ctypes.byref(p), _stream(stream, dev)))
    return g


def _norm_params(q, k, wq, wk, kind, eps, cos, sin, positions, interleaved):
    import torch

    B, L, Hq, d = q.shape
    Hk = k.shape[2]
    qs = _tokens(q, (B, L, Hq, d), "q", q.dtype)
    ks = _tokens(k, (B, L, Hk, d), "k", q.dtype)
    for t, name in ((wq, "wq"), (wk, "wk")):
        if t is not None:
            _need(t, (d,), name, torch.float32)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    rot = P = 0
    if cos is not None:
        P, half = cos.shape
        rot = 2 * half
        _need(cos, (P, half), "cos", torch.float32)
        _need(sin, (P, half), "sin", torch.float32)
    if positions is not None:
        _need(positions, (B, L), "positions", torch.int32)
    p = QkNormParams(B, L, Hq, Hk, d, rot, P, _b._dtype_code(q), 0, q.data_ptr(), k.data_ptr(), qs, ks, _addr(wq),
                     _addr(wk), _addr(cos), _addr(sin), _addr(positions))
    p.eps = eps
    if kind not in _NORM_KINDS:
        raise ValueError("kind is 'rms' or 'l2' (got %r)" % (kind,))
    p.norm_kind = _NORM_KINDS[kind]
    p.interleaved = int(bool(interleaved))
    return p


def ssm_qk_norm_fwd(q, k, *, wq=None, wk=None, kind="rms", eps=1e-6, cos=None, sin=None, positions=None,
                    interleaved=False, q_out=None, k_out=None, out_dtype=None, stream=None):
    """Norms of q (B, L, Hq, d) and k (B, L, Hk, d) for each head, then the
    position rotation of the first 2 * cos.shape[1] entries; returns (q_out, k_out).

    kind "rms" or "l2"; wq, wk: (d,) float32 or None; cos, sin: (positions, pairs)
    float32 tables or None; positions: (B, L) int32, None for 0 .. L - 1;
    interleaved turns neighbours instead of halves. Outputs are allocated
    (float32 unless ``out_dtype`` says bfloat16) when not given.
    """
    import torch

    lib = _b.load_library()
    dt = out_dtype or torch.float32
    if q_out is None:
        q_out = _out(q, dt, stream)
    if k_out is None:
        k_out = _out(k, q_out.dtype, stream)
    p = _norm_params(q, k, wq, wk, kind, eps, cos, sin, positions, interleaved)
    _need(q_out, q.shape, "q_out", q_out.dtype)
    _need(k_out, k.shape, "k_out", q_out.dtype)
    p.out_dtype, p.q_out, p.k_out = _b._dtype_code(q_out), q_out.data_ptr(), k_out.data_ptr()
    _b._check(lib.ssm_qk_norm_fwd(ctypes.byref(p), _stream(stream, q.device)))
    return q_out, k_out


def ssm_qk_norm_bwd(q, k, dq_out, dk_out, *, wq=None, wk=None, kind="rms", eps=1e-6, cos=None, sin=None,
                    positions=None, interleaved=False, grad_dtype=None, want_dw=True, workspace=None, stream=None):
    """Gradients of ssm_qk_norm_fwd for the same inputs and the outputs'
    gradients. Returns a dict with dq, dk in ``grad_dtype`` (float32 by default)
    and float32 dwq, dwk (d,) (None without ``want_dw``)."""
    import torch

    lib = _b.load_library()
    dt = grad_dtype or torch.float32
    g = dict(dq=_out(q, dt, stream), dk=_out(k, dt, stream))
    for name in ("dwq", "dwk"):
        g[name] = _b._result(q.shape[3], torch.float32, q.device, stream) if want_dw else None
    p = _norm_params(q, k, wq, wk, kind, eps, cos, sin, positions, interleaved)
    _need(dq_out, q.shape, "dq_out", q.dtype)
    _need(dk_out, k.shape, "dk_out", q.dtype)
    p.out_dtype = _b._dtype_code(g["dq"])
    p.dq_out, p.dk_out, p.dq, p.dk = dq_out.data_ptr(), dk_out.data_ptr(), g["dq"].data_ptr(), g["dk"].data_ptr()
    p.dwq, p.dwk = _addr(g["dwq"]), _addr(g["dwk"])
    workspace = _workspace(lib.ssm_qk_norm_bwd_workspace_size, p, workspace, q.device, stream)
    _b._check(lib.ssm_qk_norm_bwd(ctypes.byref(p), _stream(stream, q.device)))
    return g

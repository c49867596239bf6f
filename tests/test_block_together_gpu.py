"""The recurrence and the norms around it as a model uses them: blocks in a row, trained through torch.autograd, served token
by token, in a captured graph and on several streams."""
import numpy as np
import pytest

from oracle import block as ob
from oracle import glr as og
from selective_state_space_67_amd import workloads as wl

from delta_helpers import check, device
from glr_helpers import STATE, call, glr_inputs, on_device, wide

pytestmark = pytest.mark.gpu

WIDTH, CHANNELS, HEADS = 96, 128, 2


def functions():
    """The operators as autograd functions."""
    import torch

    import selective_state_space_67_amd as ssm

    class Recurrence(torch.autograd.Function):
        @staticmethod
        def forward(ctx, u, dt, i, A, dt_bias, in_bias, reset):
            ctx.save_for_backward(u, dt, i, A, dt_bias, in_bias, reset)
            return ssm.ssm_glr_fwd(u, dt, A, dt_bias=dt_bias, in_raw=i, in_bias=in_bias, reset=reset)

        @staticmethod
        def backward(ctx, dout):
            u, dt, i, A, dt_bias, in_bias, reset = ctx.saved_tensors
            g = ssm.ssm_glr_bwd(u, dt, A, dout.contiguous(), dt_bias=dt_bias, in_raw=i, in_bias=in_bias, reset=reset,
                                want_dh0=False)
            return g["du"], g["d_dt_raw"], g["din_raw"], g["dA"], g["d_dt_bias"], g["din_bias"], None

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, z, w):
            ctx.save_for_backward(x, z, w)
            return ssm.ssm_gated_norm_fwd(x, z, w=w)

        @staticmethod
        def backward(ctx, dout):
            x, z, w = ctx.saved_tensors
            g = ssm.ssm_gated_norm_bwd(x, z, dout.contiguous(), w=w)
            return g["dx"], g["dz"], g["dw"]

    class Join(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y, x, w, w_post, gate):
            ctx.save_for_backward(y, x, w, w_post, gate)
            return ssm.ssm_block_norm_fwd(y, x, w=w, post=True, w_post=w_post, gate=gate, scale=0.5)

        @staticmethod
        def backward(ctx, dout, dx_out):
            y, x, w, w_post, gate = ctx.saved_tensors
            g = ssm.ssm_block_norm_bwd(y, x, dout.contiguous(), dx_out.contiguous(), w=w, post=True, w_post=w_post, gate=gate,
                                       scale=0.5)
            return g["dy"], g["dx"], g["dw"], g["dw_post"], g["dgate"]

    return Recurrence.apply, Gated.apply, Join.apply


def weights(dtype, dev, seed=0):
    import torch

    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    w = dict(A=torch.log(0.9 + 0.099 * torch.rand(CHANNELS, generator=gen, dtype=torch.float64)), dt_bias=n(CHANNELS),
             in_bias=n(CHANNELS), gate=0.3 * n(WIDTH), w_gated=1 + 0.1 * n(CHANNELS // HEADS), w=1 + 0.1 * n(WIDTH),
             w_post=1 + 0.1 * n(WIDTH), back=n(CHANNELS, WIDTH) / CHANNELS ** 0.5,
             project=n(WIDTH, 4 * CHANNELS) / WIDTH ** 0.5)
    return {k: v.to(dtype).to(dev).requires_grad_(True) for k, v in w.items()}


def model(x, first, w, reset, recurrence, gated, join, blocks=2):
    """Blocks in a row on the residual stream x, whose normed form is `first`; the last norm's output."""
    n = first
    for _ in range(blocks):
        u, dt, i, z = (n @ w["project"]).split(CHANNELS, -1)
        h = recurrence(u, dt, i, w["A"], w["dt_bias"], w["in_bias"], reset)
        heads = h.unflatten(-1, (HEADS, -1))
        y = gated(heads, z.unflatten(-1, (HEADS, -1)), w["w_gated"]).flatten(2) @ w["back"]
        n, x = join(y, x, w["w"], w["w_post"], w["gate"])
    return n


def plain_functions():
    """The same from torch's elementary operations (for float64 on the CPU)."""
    import torch

    def norm(v):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + float(np.float32(1e-6)))

    def recurrence(u, dt, i, A, dt_bias, in_bias, reset):
        g = A * torch.sigmoid(dt + dt_bias)
        on = (reset != 0)[..., None]
        a = torch.where(on, torch.zeros_like(g), torch.exp(g))
        c = torch.where(on, torch.ones_like(g), torch.sqrt(-torch.expm1(2 * g)))
        b, h, out = c * torch.sigmoid(i + in_bias) * u, torch.zeros_like(u[:, 0]), []
        for t in range(u.shape[1]):
            h = a[:, t] * h + b[:, t]
            out.append(h)
        return torch.stack(out, 1)

    def gated(x, z, w):
        return w * norm(x) * z * torch.sigmoid(z)

    def join(y, x, w, w_post, gate):
        x = x + 0.5 * gate * w_post * norm(y)
        return w * norm(x), x

    return recurrence, gated, join


def test_blocks_train_as_in_float64():
    """Loss gradients of two blocks against automatic differentiation of the plain forms in float64.

    Each operator's outputs and gradients are held to 1e-5 .. 1e-4 of their size by their own tests and products in float32 add
    1e-6; through two blocks and back these add up and the norms hand them on at their own size: 1e-3 of the root mean square.
    """
    import torch

    B, L = 2, 300
    rng = np.random.default_rng(0)
    data = {k: rng.standard_normal((B, L, WIDTH)) for k in ("x", "first", "target")}
    reset = np.zeros((B, L), np.uint8)
    reset[0, 0] = reset[0, 120] = reset[1, 255] = 1
    grads = {}
    for dtype, dev, fns in ((torch.float32, device(), functions()), (torch.float64, "cpu", plain_functions())):
        w = weights(dtype, dev)
        t = {k: torch.from_numpy(v).to(dtype).to(dev) for k, v in data.items()}
        x = t["x"].requires_grad_(True)
        out = model(x, t["first"], w, torch.from_numpy(reset).to(dev), *fns)
        ((out - t["target"]).square().mean()).backward()
        grads[dtype] = {k: v.grad.double().cpu() for k, v in dict(w, x=x).items()}
        grads[dtype]["out"] = out.detach().double().cpu()
    for k, ref in grads[torch.float64].items():
        gap = (grads[torch.float32][k] - ref).abs().max() / ref.square().mean().sqrt()
        assert gap < 1e-3, (k, float(gap))


def test_serving_agrees_with_the_whole_sequence():
    """A prompt, then windows of tokens with the state kept: each step's outputs are the whole sequence's."""
    import torch

    import selective_state_space_67_amd as ssm

    B, L = 3, 350
    x = glr_inputs(B, L, CHANNELS, wl.BF16, seed=4, z=True)
    t = on_device(x, device())
    a, k = call(t)
    whole = ssm.ssm_glr_fwd(*a, **k)
    state = torch.zeros(B, CHANNELS, device=device())
    parts, at = [], 0
    for n in (300, 1, 1, 4, 1, 40, 3):
        s = {m: t[m][:, at:at + n].contiguous() for m in ("u", "dt_raw", "in_raw", "z")}
        b, kw = call({**t, **s})
        if n > 8:
            last = torch.empty_like(state)
            parts.append(ssm.ssm_glr_fwd(*b, h0=state, h_last=last, **kw))
            state = last
        else:
            parts.append(ssm.ssm_glr_update(state, *b, **kw))
        at += n
    torch.cuda.synchronize()
    ref, rh = og.glr_fwd(**wide(x))
    check(torch.cat(parts, 1), ref, STATE, "served")
    check(whole, ref, STATE, "whole")
    check(state, rh, STATE, "state")


def test_all_of_them_in_a_graph():
    """Captured once, replayed three times with eager work of the same calls between, bit for bit the eager results."""
    import torch

    import selective_state_space_67_amd as ssm

    x = glr_inputs(2, 700, 130, wl.BF16, seed=5, z=True, state=True, resets=[(0, 70), (1, 640)])
    t = on_device(x, device())
    a, k = call(t)
    one = {m: t[m][:, :1].contiguous() for m in ("u", "dt_raw", "in_raw", "z")}
    b, kb = call({**t, **one})
    w, gate = torch.rand(130, device=device()), torch.rand(2, 130, device=device())
    stream = torch.randn(2, 700, 130, device=device())
    h = t["h0"].clone()

    def work():
        h.copy_(t["h0"])
        last = torch.empty_like(h)
        out = ssm.ssm_glr_fwd(*a, reset=t["reset"], h0=t["h0"], h_last=last, out_dtype=torch.bfloat16, **k)
        g = ssm.ssm_glr_bwd(*a, t["dout"], reset=t["reset"], h0=t["h0"], dh_last=t["dh_last"], **k)
        heads = out.unflatten(-1, (2, 65))
        y = ssm.ssm_gated_norm_fwd(heads, t["z"].unflatten(-1, (2, 65)), out_dtype=torch.bfloat16)
        gn = ssm.ssm_gated_norm_bwd(heads, t["z"].unflatten(-1, (2, 65)), y, w=w[:65].contiguous())
        n, s = ssm.ssm_block_norm_fwd(y.flatten(2), stream, w=w, post=True, gate=gate)
        gb = ssm.ssm_block_norm_bwd(y.flatten(2), stream, t["dout"], s, w=w, post=True, gate=gate)
        steps = [ssm.ssm_glr_update(h, *b, **kb) for _ in range(3)]
        both = [v for d in (g, gn, gb) for v in d.values() if v is not None]
        return [out, last, y, n, s, h] + steps + both

    ref = [r.clone() for r in work()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for rep in range(3):
        if rep:
            again = ssm.ssm_glr_fwd(*a, reset=t["reset"], h0=t["h0"], out_dtype=torch.bfloat16, **k)
            torch.cuda.synchronize()
            assert torch.equal(again, ref[0])
        graph.replay()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(got, ref)):
            assert torch.equal(p, q), (rep, i)


def test_calls_at_once_on_several_streams():
    """Forwards in pieces and backwards on four streams at the same time, each with memory of its own, give the bits of calls in turn."""
    import torch

    import selective_state_space_67_amd as ssm

    inputs = [on_device(glr_inputs(1, 20000 + 1000 * i, 70, wl.BF16, seed=i, z=True, state=True), device()) for i in range(4)]

    def run(t, stream):
        a, k = call(t)
        return [ssm.ssm_glr_fwd(*a, h0=t["h0"], stream=stream, **k),
                ssm.ssm_glr_bwd(*a, t["dout"], h0=t["h0"], stream=stream, **k)["dA"]]

    ref = [run(t, None) for t in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    for _ in range(3):
        got = [run(t, s) for t, s in zip(inputs, streams)]
        torch.cuda.synchronize()
        for p, q in zip(got, ref):
            assert all(torch.equal(x, y) for x, y in zip(p, q))


def test_a_workspace_is_used_again():
    """The same workspace for one call after another, whatever it holds; one that is too small is replaced."""
    import torch

    import selective_state_space_67_amd as ssm

    x = glr_inputs(1, 3000, 70, wl.F32, seed=8, state=True)
    t = on_device(x, device())
    a, k = call(t)
    ref = ssm.ssm_glr_fwd(*a, h0=t["h0"], **k)
    for fill in (0, 255, 17):
        ws = torch.full((1 << 22,), fill, dtype=torch.uint8, device=device())
        for _ in range(2):
            assert torch.equal(ssm.ssm_glr_fwd(*a, h0=t["h0"], workspace=ws, **k), ref)
    assert torch.equal(ssm.ssm_glr_fwd(*a, h0=t["h0"], workspace=ws[:256], **k), ref)
    check(ref, og.glr_fwd(**wide(x))[0], STATE, "out")


def test_rows_behind_the_last_are_left_alone():
    """Outputs that are parts of larger buffers: nothing before or behind them is written."""
    import torch

    import selective_state_space_67_amd as ssm

    for B, L, D in ((1, 5, 70), (2, 37, 70), (1, 1003, 70)):
        t = on_device(glr_inputs(B, L, D, wl.BF16, seed=L), device())
        a, k = call(t)
        n = B * L * D
        buf = torch.full((n + 2 * 512,), 7.0, device=device(), dtype=torch.bfloat16)
        out = buf[512:512 + n].view(B, L, D)
        ssm.ssm_glr_fwd(*a, out=out, **k)
        y = t["u"].unflatten(-1, (2, 35))
        buf2 = buf.clone()
        ssm.ssm_gated_norm_fwd(y, y, out=buf2[512:512 + n].view(B, L, 2, 35))
        buf3 = buf.clone()
        ssm.ssm_block_norm_fwd(t["u"], out=buf3[512:512 + n].view(B, L, D))
        torch.cuda.synchronize()
        for b in (buf, buf2, buf3):
            assert bool((b[:512] == 7).all()) and bool((b[512 + n:] == 7).all())
        check(buf3[512:512 + n].view(B, L, D), ob.block_norm(wl.widen(wl_store(t["u"])), eps=1e-6)[0], 3e-6, "out", bf16=True)


def wl_store(t):
    return t.float().cpu().numpy().astype(np.float32)


def test_long_offsets():
    """Rows whose place in memory passes 2^31 elements (a slice of a wide projection) and 2^32 bytes."""
    import torch

    import selective_state_space_67_amd as ssm

    L, stride, D = 600, 4_000_000, 66
    packed = torch.empty((1, L, stride), device=device(), dtype=torch.bfloat16)
    s = {}
    x = glr_inputs(1, L, D, wl.BF16, seed=11)
    t = on_device(x, device())
    for j, n in enumerate(("u", "dt_raw", "in_raw")):
        s[n] = packed[..., j * D:(j + 1) * D]
        s[n].copy_(t[n])
    a, k = call(t)
    b, m = call({**t, **s})
    assert torch.equal(ssm.ssm_glr_fwd(*a, **k), ssm.ssm_glr_fwd(*b, **m))
    g, f = ssm.ssm_glr_bwd(*a, t["dout"], **k), ssm.ssm_glr_bwd(*b, t["dout"], **m)
    y = s["u"].unflatten(-1, (1, D))
    z = s["in_raw"].unflatten(-1, (1, D))
    gated = ssm.ssm_gated_norm_fwd(y, z), ssm.ssm_gated_norm_fwd(y.contiguous(), z.contiguous())
    joined = ssm.ssm_block_norm_fwd(s["u"]), ssm.ssm_block_norm_fwd(t["u"])
    torch.cuda.synchronize()
    assert all(torch.equal(g[n], f[n]) for n in g if g[n] is not None)
    assert torch.equal(*gated) and all(torch.equal(p, q) for p, q in zip(*joined))

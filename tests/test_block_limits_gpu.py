"""The block norm with a gate for each of very many sequences, against torch in float64."""
import numpy as np
import pytest

from delta_helpers import device
from test_block_norm_gpu import FWD, GRAD, SUM

pytestmark = pytest.mark.gpu


def close(got, want, tol, name):
    bound = tol * (want.square().mean().sqrt() + want.abs()) + 1e-30
    assert bool(((got.double() - want).abs() <= bound).all()), name


# the sums of dgate, dw (and dw_post) together have a few workgroups more than a launch has room for; dgate's alone fit
@pytest.mark.parametrize("B,D,post", [(16383, 8192, False), (8191, 16384, True)])
def test_sums_of_many_gates(B, D, post):
    import torch

    from selective_state_space_67_amd import ssm_block_norm_bwd

    dev = device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(D)
    y, dout = (torch.randn(B, 1, D, generator=gen, device=dev, dtype=torch.bfloat16) for _ in range(2))
    gate = torch.randn(B, D, generator=gen, device=dev)
    w, w_post = 0.5 + torch.rand(D, generator=gen, device=dev), 0.5 + torch.rand(D, generator=gen, device=dev)
    eps = float(np.float32(1e-5))
    print(B, D, post, flush=True)
    g = ssm_block_norm_bwd(y, None, dout, w=w, post=post, w_post=w_post if post else None, gate=gate, scale=0.5, eps=eps)
    torch.cuda.synchronize()
    dw, dwp = torch.zeros(D, device=dev, dtype=torch.float64), torch.zeros(D, device=dev, dtype=torch.float64)
    wd, wp = w.double(), w_post.double() if post else torch.ones(D, device=dev, dtype=torch.float64)
    for i in range(0, B, 1024):
        a, d, k = y[i:i + 1024, 0].double(), dout[i:i + 1024, 0].double(), 0.5 * gate[i:i + 1024].double()
        ry = torch.rsqrt(a.square().mean(-1, keepdim=True) + eps) if post else 1.0
        m = a * ry * wp
        s = k * m
        r = torch.rsqrt(s.square().mean(-1, keepdim=True) + eps)
        n = s * r
        dw += (d * n).sum(0)
        dX = r * (d * wd - n * (d * wd * n).mean(-1, keepdim=True))
        close(g["dgate"][i:i + 1024], 0.5 * m * dX, GRAD, "dgate of rows from %d" % i)
        dwp += (dX * k * a * ry).sum(0)
    close(g["dw"], dw, SUM, "dw")
    if post:
        close(g["dw_post"], dwp, SUM, "dw_post")


def test_forward_of_more_gates_than_the_backward_sums():
    import torch

    from selective_state_space_67_amd import ssm_block_norm_fwd

    B, D, dev = 8192, 16384, device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(1)
    y = torch.randn(B, 1, D, generator=gen, device=dev, dtype=torch.bfloat16)
    gate = torch.randn(B, D, generator=gen, device=dev)
    print(B, D, flush=True)
    out, x = ssm_block_norm_fwd(y, None, gate=gate, scale=0.5)
    torch.cuda.synchronize()
    for i in range(0, B, 1024):
        s = 0.5 * gate[i:i + 1024].double() * y[i:i + 1024, 0].double()
        close(x[i:i + 1024, 0], s, FWD, "x_out of rows from %d" % i)
        close(out[i:i + 1024, 0], s * torch.rsqrt(s.square().mean(-1, keepdim=True) + float(np.float32(1e-6))), FWD,
              "out of rows from %d" % i)

"""Scan calls with stream=: the current stream goes on allocating and writing while they wait and run."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["fwd", "bwd", "update"])
def test_the_current_stream_takes_none_of_a_calls_memory(name):
    import torch

    import selective_state_space_67_amd as ssm

    torch.manual_seed(5)
    r = lambda *s: torch.randn(*s, device="cuda:0")  # noqa: E731
    B, D, L, N = 1, 64, 8192, 16  # split into pieces, so that the forward has a workspace too
    u, dt, A, Bm, Cm, dout = r(B, D, L), r(B, D, L) - 4, -r(D, N).abs(), r(B, L, N), r(B, L, N), r(B, D, L)
    h, u1, B1 = r(B, D, N), r(B, D), r(B, N)
    call = {"fwd": lambda **kw: [ssm.ssm_scan_fwd(u, dt, A, Bm, Cm, **kw)],
            "bwd": lambda **kw: [g for g in ssm.ssm_scan_bwd(u, dt, A, Bm, Cm, dout, **kw).values() if g is not None],
            "update": lambda **kw: [ssm.ssm_state_update(h, u1, u1, A, B1, B1, **kw)]}[name]
    start = h.clone()
    want = [w.clone() for w in call()]
    h.copy_(start)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some milliseconds during which the call waits
    print(name, flush=True)
    got = call(stream=side)
    taken = []
    for size in (1 << 12, 1 << 16, 1 << 18, 1 << 20, 1 << 21, 1 << 22, 1 << 24, 1 << 26):
        for _ in range(4):
            taken.append(torch.empty(size, dtype=torch.uint8, device="cuda:0").fill_(255))
    del taken
    side.synchronize()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)

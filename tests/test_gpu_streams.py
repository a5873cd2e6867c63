"""Calls on a stream of the caller's: their outputs come from that stream's memory, never from a block that work still
pending on another stream may be using, and stay the caller's as long as its own stream reads them."""
import pytest
import torch

from state_space_model_scan_gb300 import api

pytestmark = pytest.mark.gpu
N16 = torch.bfloat16


def randn(*s, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(sum(s))
    return (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)


def scan_args(L=512, Dm=1024, N=16):
    return (randn(1, L, Dm, dtype=N16), randn(1, L, Dm, dtype=N16), -torch.exp(randn(Dm, N, scale=0.1)), randn(1, L, 1, N, dtype=N16),
            randn(1, L, 1, N, dtype=N16))


def new_calls():
    """Name, call(stream) -> tensors.  Calls that update something in place give the same output every time: states that
    a step of 50 forgets, windows that the taps do not see."""
    a = scan_args()
    dy = randn(1, 512, 1024, dtype=N16)
    n, H, P, N = 256, 40, 64, 16
    pool = torch.zeros(n, H, P, N, device="cuda")
    step = (randn(n, H, P, dtype=N16), 50 + randn(n, H), -1 - randn(H).abs(), randn(n, 1, N, dtype=N16), randn(n, 1, N, dtype=N16))
    pool2 = torch.zeros(n, 4096, N, device="cuda")
    step2 = (randn(n, 4096, dtype=N16), (50 + randn(n, 4096)).to(N16), -1 - randn(4096, N).abs(), step[3], step[4])
    u, win = randn(1, 1024, 1024, dtype=N16), torch.zeros(1, 3, 1024, dtype=N16, device="cuda")
    u1, win1 = randn(512, 2048, dtype=N16), torch.zeros(512, 3, 2048, dtype=N16, device="cuda")
    w, w1 = randn(1024, 4), randn(2048, 4)
    w[:, :3] = w1[:, :3] = 0
    return {
        "selective_scan_forward": lambda s: api.selective_scan_forward(*a, keep_chunk_states=True, stream=s),
        "selective_scan_backward": lambda s: tuple(api.selective_scan_backward(*a, dy, stream=s).values()),
        "ssd_step": lambda s: (api.ssd_step(pool, *step, stream=s),),
        "selective_scan_step": lambda s: (api.selective_scan_step(pool2, *step2, stream=s),),
        "conv1d_prompt": lambda s: (api.conv1d_prompt(u, w, None, win, stream=s),),
        "conv1d_step": lambda s: (api.conv1d_step(u1, w1, None, win1, stream=s),),
    }


NEW = ["selective_scan_forward", "selective_scan_backward", "ssd_step", "selective_scan_step", "conv1d_prompt", "conv1d_step"]


def scan_calls():
    """The same for the calls of the per-head scan, the normalisation, the plain convolution and the complex scan."""
    L, H, P, G, N = 512, 16, 64, 1, 128
    a = (randn(1, L, H, P, dtype=N16), randn(1, L, H), -torch.exp(randn(H)), randn(1, L, G, N, dtype=N16), randn(1, L, G, N, dtype=N16))
    y, nw = randn(512, 2048, dtype=N16), randn(2048)
    _, rstd = api.gated_norm_forward(y, nw, 1024, z=y)
    u, w = randn(1, 1024, 1024, dtype=N16), randn(1024, 4)
    c = [randn(1, 256, 8, 64, 2).view(1, 256, 8, 64, 2) for _ in range(3)]
    c = [torch.view_as_complex(t) for t in c]
    cA, cdt = torch.complex(-torch.exp(randn(8)), randn(8)), randn(1, 256, 8)
    return {
        "ssd_forward": lambda s: api.ssd_forward(*a, stream=s),
        "ssd_backward": lambda s: tuple(api.ssd_backward(*a, a[0], stream=s).values()),
        "gated_norm_forward": lambda s: api.gated_norm_forward(y, nw, 1024, z=y, stream=s),
        "gated_norm_backward": lambda s: api.gated_norm_backward(y, nw, rstd, y, 1024, z=y, stream=s),
        "conv1d_forward": lambda s: (api.conv1d_forward(u, w, None, None, True, s),),
        "conv1d_backward": lambda s: api.conv1d_backward(u, w, u, stream=s)[:2],
        "complex_ssd_forward": lambda s: (api.complex_ssd_forward(c[0], cA, c[1], c[2], cdt, stream=s),),
    }


SCAN = ["ssd_forward", "ssd_backward", "gated_norm_forward", "gated_norm_backward", "conv1d_forward", "conv1d_backward", "complex_ssd_forward"]


def spans(ts):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in ts]


def apart(a, b):
    return all(x1 <= y0 or y1 <= x0 for x0, x1 in a for y0, y1 in b)


def check_outputs(call):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    want = [t.clone() for t in call(None)]
    # blocks that the current stream has freed, of the outputs' very sizes
    mine = [torch.empty_like(t) for t in want]
    freed = spans(mine)
    torch.cuda.synchronize()
    del mine
    got = call(side)
    assert apart(freed, spans(got))
    torch.cuda.current_stream().wait_stream(side)
    for t, v in zip(got, want):
        assert torch.equal(t, v)
    # given back while the current stream still has to read them, they are not handed out for the next call
    torch.cuda.synchronize()
    del t, v
    held = spans(got)
    torch.cuda._sleep(200_000_000)                                 # a tenth of a second of the current stream
    keep = [g.clone() for g in got]
    del got
    again = call(side)
    assert apart(held, spans(again))
    torch.cuda.synchronize()
    for t, v in zip(keep, want):
        assert torch.equal(t, v)


@pytest.mark.parametrize("name", NEW)
def test_outputs_come_from_the_streams_own_memory(name):
    check_outputs(new_calls()[name])


@pytest.mark.parametrize("name", NEW)
def test_default_stream_given_inside_another(name):
    call = new_calls()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(torch.cuda.default_stream())
    torch.cuda.synchronize()
    for t, v in zip(got, want):
        assert torch.equal(t, v)


@pytest.mark.parametrize("name", SCAN)
def test_scan_outputs_come_from_the_streams_own_memory(name):
    check_outputs(scan_calls()[name])


def test_workspace_grows_while_another_stream_uses_it():
    """The buffer that a growing workspace gives up is not handed out while a stream that has worked in it may still do so."""
    ws, side = api.Workspace(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = spans([ws.get(8 << 20)])
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        ws.get(8 << 20).fill_(1)
    ws.get(16 << 20)
    assert apart(old, spans([torch.empty(8 << 20, dtype=torch.uint8, device="cuda")]))
    torch.cuda.synchronize()

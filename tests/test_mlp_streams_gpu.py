"""The MLP operators on a stream given by argument, while the caller's stream
goes on allocating and writing."""
import pytest
import torch

from tests.test_mlp_gpu import gen, rows, weights
from w4a8_quantized_gemm_channel_b200 import native

pytestmark = pytest.mark.gpu

DELAY = 20_000_000      # cycles, some 10 ms: the given stream starts well after the caller's next allocations


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    native.get_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert native.get_device_status() == 0


def calls(m, dt):
    d, f = 320, 900
    rnd = gen(m)
    p = {}
    for name, (n, k) in dict(g=(f, d), u=(f, d)).items():
        _, sw, wp = weights(rnd, n, k)
        p[name] = (wp, sw)
    x, dh = rows(rnd, m, d, dt), rnd(m, f, std=0.01).to(dt)
    _, g, u = native.w4a8_glu(x, *p["g"], *p["u"], save=True)
    return {
        "linear": lambda **kw: native.w4a8_linear_act(x, *p["g"], act="gelu", save=True, **kw),
        "glu": lambda **kw: native.w4a8_glu(x, *p["g"], *p["u"], save=True, **kw),
        "linear_grad": lambda **kw: native.w4a8_linear_act_grad(dh, *p["g"], d, act="silu", z=g, bias_grad=True, **kw),
        "glu_grad": lambda **kw: native.w4a8_glu_grad(dh, g, u, *p["g"], *p["u"], d, bias_grad=True, **kw),
    }


@pytest.mark.parametrize("op", ["linear", "glu", "linear_grad", "glu_grad"])
@pytest.mark.parametrize("m,io", [(3, torch.float32), (300, torch.bfloat16), (300, torch.float32)])
def test_call_on_a_given_stream(op, m, io):
    """The call is still waiting on its stream when the caller's stream takes
    and overwrites memory, as much as the call has released."""
    call = calls(m, io)[op]
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(DELAY)
        got = call(stream=s)
        noise = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in [1 << b for b in range(10, 25)] * 2]
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del noise


def test_results_outlive_their_last_use_on_the_callers_stream():
    """A result made on a given stream and released while the caller's stream
    still reads it is not overwritten by that stream's next call."""
    call = calls(300, torch.float32)["glu"]
    want = call()[0].clone()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = call(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(DELAY)
        seen = got[0].clone()              # behind the delay
        del got
        with torch.cuda.stream(s):
            junk = [torch.full_like(want, float("nan")) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(seen, want)
        del junk


def test_given_workspace_and_outputs_are_used():
    x = torch.randn(40, 64, device="cuda")
    _, sw, wp = weights(gen(1), 48, 64)
    ws = torch.empty(native.act_workspace_size(40, 64, 48), dtype=torch.uint8, device="cuda")
    y = torch.empty(40, 48, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = native.w4a8_linear_act(x, wp, sw, y=y, workspace=ws, stream=s)
    s.synchronize()
    assert out is y and torch.equal(y, native.w4a8_linear_act(x, wp, sw))


def test_stream_in_a_capture():
    """A given stream that belongs to a capture records the call there."""
    call = calls(40, torch.bfloat16)["glu_grad"]
    want = call()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = call(stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)

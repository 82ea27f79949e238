"""The binding's `stream` argument, on the host: whatever a call allocates is
allocated with that stream current, and the kernels are enqueued there."""
import contextlib

import pytest
import torch

from w4a8_quantized_gemm_channel_b200 import native


class FakeStream:
    device = torch.device("cpu")
    cuda_stream = 0x5EED


class CallerStream:
    cuda_stream = 0


class FakeLib:
    """Every function succeeds; sizes are 64; calls and the current stream are recorded."""

    def __init__(self, now):
        self.now, self.calls = now, []

    def __getattr__(self, name):
        def fn(*args):
            if name.endswith(("_size", "_ld", "_parts", "_groups")):
                return 64
            self.calls.append((name, self.now[0], getattr(args[-1], "value", args[-1])))
            return 0
        return fn


@pytest.fixture
def world(monkeypatch):
    now, made = ["caller"], []

    @contextlib.contextmanager
    def entered(s):
        now.append(now[0])
        now[0] = "given" if isinstance(s, FakeStream) else "caller"
        yield
        now[0] = now.pop()

    def noted(make):
        def f(*a, **k):
            t = make(*a, **k)
            made.append(now[0])
            return t
        return f

    lib = FakeLib(now)
    monkeypatch.setattr(native, "lib", lib)
    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream() if now[0] == "given" else CallerStream())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream",
                        lambda dev: FakeStream.cuda_stream if now[0] == "given" else 0, raising=False)
    monkeypatch.setattr(torch, "empty", noted(torch.empty))
    monkeypatch.setattr(torch.Tensor, "new_empty", noted(torch.Tensor.new_empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    monkeypatch.setattr(native, "_rows_in", lambda t, name: (*t.shape, t.stride(0), -1))
    return lib, made


X, WP, SW, DY = torch.zeros(2, 8), torch.zeros(4, 16, dtype=torch.uint8), torch.ones(4), torch.zeros(2, 4)
MLP = {
    "w4a8_linear_act": dict(x=X, wp=WP, sw=SW, save=True),
    "w4a8_glu": dict(x=X, wg=WP, sg=SW, wu=WP, su=SW, save=True),
    "w4a8_linear_act_grad": dict(dy=DY, wp=WP, sw=SW, k=8, bias_grad=True),
    "w4a8_glu_grad": dict(dh=DY, g=DY, u=DY, wg=WP, sg=SW, wu=WP, su=SW, k=8, bias_grad=True),
}
W, XQ, SX, ZP = torch.zeros(8, 4), torch.zeros(2, 16, dtype=torch.int8), torch.ones(2), torch.zeros(4, dtype=torch.int32)
W8 = torch.zeros(4, 16, dtype=torch.int8)
CALLS = dict(MLP,
    w4_quantize_pack=dict(w=W), a8_quantize_rows=dict(x=X), w8_quantize=dict(w=W), w4z_quantize_pack=dict(w=W),
    w4g_quantize_pack=dict(w=W),
    w4a8_linear=dict(x=X, wp=WP, sw=SW), w4a8_linear_q=dict(xq=XQ, sx=SX, k=8, wp=WP, sw=SW),
    w4a8_linear_chain=dict(x=X, wp=WP, sw=SW), w4a8_linear_noalloc=dict(x=X, wp=WP, sw=SW),
    w4a8_linear_grouped=dict(problems=[(X, WP, SW, None), (X, WP, SW, SW)]),
    w8a8_linear=dict(x=X, wq=W8, sw=SW), w8a8_linear_q=dict(xq=XQ, sx=SX, k=8, wq=W8, sw=SW),
    w4z_linear=dict(x=X, wp=WP, sa=SW, zp=ZP), w4z_linear_q=dict(xq=XQ, sx=SX, k=8, wp=WP, sa=SW, zp=ZP),
    w4g_linear=dict(x=X, wp=WP, sa=SW, zp=ZP), w4g_linear_q=dict(xq=XQ, sx=SX, k=8, wp=WP, sa=SW, zp=ZP))


@pytest.mark.parametrize("name", CALLS)
def test_allocations_belong_to_the_given_stream(world, name):
    lib, made = world
    getattr(native, name)(**CALLS[name], stream=FakeStream())
    assert made and set(made) == {"given"}
    assert [c[1:] for c in lib.calls] == [("given", FakeStream.cuda_stream)]


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one_is_used(world, name):
    lib, made = world
    getattr(native, name)(**CALLS[name])
    assert made and set(made) == {"caller"} and lib.calls[0][1] == "caller"

"""The layer's calls on a stream given by argument, while the caller's stream
goes on allocating and writing (the MLP operators: test_mlp_streams_gpu.py)."""
import pytest
import torch

from w4a8_quantized_gemm_channel_b200 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def calls():
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    w, x = torch.randn(500, 260, generator=g, device="cuda"), torch.randn(70, 500, generator=g, device="cuda")
    wp, sw = native.w4_quantize_pack(w)
    wq, sw8 = native.w8_quantize(w)
    wz, sz, zz = native.w4z_quantize_pack(w)
    wg, sg, zg = native.w4g_quantize_pack(w)
    xq, sx = native.a8_quantize_rows(x)
    return {
        "pack": lambda **kw: native.w4_quantize_pack(w, **kw),
        "rows": lambda **kw: native.a8_quantize_rows(x, **kw),
        "linear": lambda **kw: (native.w4a8_linear(x, wp, sw, **kw),),
        "linear_q": lambda **kw: (native.w4a8_linear_q(xq, sx, 500, wp, sw, **kw),),
        "chain": lambda **kw: native.w4a8_linear_chain(x, wp, sw, **kw),
        "w8": lambda **kw: (native.w8a8_linear(x, wq, sw8, **kw),),
        "zero_point": lambda **kw: (native.w4z_linear(x, wz, sz, zz, **kw),),
        "group_wise": lambda **kw: (native.w4g_linear(x, wg, sg, zg, **kw),),
        "grouped": lambda **kw: native.w4a8_linear_grouped([(x[:2], wp, sw, None), (x[2:3], wp, sw, None)], **kw),
    }


@pytest.mark.parametrize("op", ["pack", "rows", "linear", "linear_q", "chain", "w8", "zero_point", "group_wise",
                                "grouped"])
def test_call_on_a_given_stream(op):
    call = calls()[op]
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = call(stream=s)
        noise = [torch.full((1 << b,), 0xFF, dtype=torch.uint8, device="cuda") for b in list(range(10, 23)) * 2]
        s.synchronize()
        # (packed rows and INT8 rows: all bytes, the padding included, are written)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del noise

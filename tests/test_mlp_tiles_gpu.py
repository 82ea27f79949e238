"""The tensor-core form's larger tiles (256 and 128 tokens; the shapes of
test_mlp_gpu.py all take 64), whole tiles in several rounds per CTA pair and
tiles shared out between pairs, with tails in every direction; and the paths
that must run. Bounds: tests/mlp_reference.py."""
import pytest
import torch

from tests import mlp_reference as ref
from tests.test_mlp_gpu import ACTS, DT, SHAPES, gen, rows, weights
from w4a8_quantized_gemm_channel_b200 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    native.get_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert native.get_device_status() == 0


def path_is(want, launches):
    assert native.last_path() == "tc" and native.last_launch_count() == launches, want


# (m, k, n, shared): plan of the call
LINEAR = [(1995, 330, 3351, False),    # 256 tokens, 112 tiles on 74 pairs
          (449, 261, 6999, False),     # 256, one round
          (267, 516, 11383, False),    # 128, 135 tiles
          (2422, 62, 257, False),      # 128, one round
          (2152, 257, 11837, True)]    # 128, shared
GLU = [(452, 700, 7129, False),        # 256, 112 tiles
       (194, 125, 7307, False),        # 256, one round
       (258, 390, 5885, False),        # 128, 138 tiles
       (67, 300, 4737, False),         # 128, one round
       (2234, 61, 11956, True)]        # 128, shared
LINEAR_GRAD = [(1755, 3885, 130, False),   # bfloat16: 256 tokens, 112 tiles; float32: 128
               (2384, 1298, 61, False),    # 256 (128), one round
               (324, 9473, 190, False),    # 128, 114 tiles
               (2370, 266, 67, False),     # 128, one round
               (2234, 61, 11956, True)]    # 128, shared
GLU_GRAD = [(1755, 3885, 131, False),      # 256 (128), 112 tiles
            (129, 11293, 9541, True),      # 256 (128), shared
            (324, 9473, 190, False),       # 128, 114 tiles
            (1227, 70, 10121, True)]       # 128, shared


def aligned(n):
    """The same tiles with rows that end on 16 bytes: outputs leave by TMA."""
    return (n, (n + 7) // 8 * 8)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n,shared", LINEAR)
def test_linear_act(io, m, k, n, shared):
    for i, n in enumerate(aligned(n)):
        rnd = gen(m + n)
        q, sw, wp = weights(rnd, n, k)
        x, r, b = rows(rnd, m, k, DT[io]), rnd(m, n, std=2.0).to(DT[io]), rnd(n)
        for act, bias, res, save in (("gelu_tanh", b, r, True), ("silu", None, None, False), ("none", b, r, False),
                                     ("gelu", b, None, True))[2 * i: 2 * i + 2]:
            got = native.w4a8_linear_act(x, wp, sw, bias=bias, act=act, residual=res, save=save, path="tc")
            path_is("linear", 3 if shared else 2)
            for t, (w, e), what in zip(got if save else (got,), ref.linear(x, q, sw, bias, act, res), "yz"):
                ref.check(t, w, e, f"{what} {act} n {n}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n,shared", GLU)
def test_glu(io, m, k, n, shared):
    for i, n in enumerate(aligned(n)):
        rnd = gen(m + n)
        (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
        x, b = rows(rnd, m, k, DT[io]), rnd(n)
        for act, bg, bu, save in (("silu", None, None, False), ("gelu", b, None, True), ("relu", None, b, True),
                                  ("gelu_tanh", b, b, False))[2 * i: 2 * i + 2]:
            got = native.w4a8_glu(x, wg, sg, wu, su, gate_bias=bg, up_bias=bu, act=act, save=save, path="tc")
            path_is("glu", 3 if shared else 2)
            for t, (w, e), what in zip(got if save else (got,), ref.glu(x, qg, sg, qu, su, bg, bu, act), "hgu"):
                ref.check(t, w, e, f"{what} {act} n {n}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n,shared", LINEAR_GRAD)
def test_linear_act_grad(io, m, k, n, shared):
    for k, act, bias in zip(aligned(k), ("gelu", "none"), (True, False)):
        rnd = gen(m + k)
        q, sw, wp = weights(rnd, n, k)
        dy, z = rnd(m, n, std=0.01).to(DT[io]), rnd(m, n, std=2.0).to(DT[io])
        got = native.w4a8_linear_act_grad(dy, wp, sw, k, act=act, z=z, bias_grad=bias, path="tc")
        path_is("linear_grad", (3 if shared else 2) + 2 * bias)
        want, db = ref.linear_grad(dy, z, q, sw, act, True)
        ref.check(got[0] if bias else got, *want, f"dx {act} k {k}")
        if bias:
            ref.check(got[1], *db[0], f"db {act}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n,shared", GLU_GRAD)
def test_glu_grad(io, m, k, n, shared):
    for k, act, bias in zip(aligned(k), ("silu", "gelu_tanh"), (False, True)):
        rnd = gen(m + k)
        (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
        dh, g, u = rnd(m, n, std=0.01).to(DT[io]), rnd(m, n, std=2.0).to(DT[io]), rnd(m, n).to(DT[io])
        got = native.w4a8_glu_grad(dh, g, u, wg, sg, wu, su, k, act=act, bias_grad=bias, path="tc")
        path_is("glu_grad", (3 if shared else 2) + (2 if bias and m > 256 else 1 if bias else 0))
        want, db = ref.glu_grad(dh, g, u, qg, sg, qu, su, act, True)
        for t, w, what in zip(got if bias else (got,), [want] + db, ("dx", "dbg", "dbu")):
            ref.check(t, *w, f"{what} {act} k {k}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_large_tiles_repeat(io):
    """Overlapped calls on the large tiles repeat the first one's bits."""
    rnd = gen(77)
    for m, k, n in ((1995, 330, 3351), (452, 700, 7129), (1755, 3885, 130)):
        (_, sg, wg), (_, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
        x, dh = rows(rnd, m, k, DT[io]), rnd(m, n, std=0.01).to(DT[io])
        _, g, u = native.w4a8_glu(x, wg, sg, wu, su, save=True)
        for call in (lambda: native.w4a8_glu(x, wg, sg, wu, su), lambda: native.w4a8_linear_act(x, wg, sg, residual=dh),
                     lambda: native.w4a8_glu_grad(dh, g, u, wg, sg, wu, su, k),
                     lambda: native.w4a8_linear_act_grad(dh, wg, sg, k)):
            first = call()
            assert all(torch.equal(first, call()) for _ in range(40))


@pytest.mark.parametrize("m,k,n", SHAPES)
def test_forced_paths_run(m, k, n):
    """The tensor-core form runs every shape, the decode form every one of at
    most 16 rows that fit a block."""
    rnd = gen(m + k + n)
    _, s, w = weights(rnd, n, k)
    x, dy = rnd(m, k), rnd(m, n)
    calls = (lambda p: native.w4a8_linear_act(x, w, s, path=p), lambda p: native.w4a8_glu(x, w, s, w, s, path=p),
             lambda p: native.w4a8_linear_act_grad(dy, w, s, k, path=p),
             lambda p: native.w4a8_glu_grad(dy, dy, dy, w, s, w, s, k, path=p))
    for i, call in enumerate(calls):
        for path in ("generic", "tc") + (("decode",) if m <= 16 and i < 2 else ()):
            call(path)
            assert native.last_path() == path
        if m > 16 or i >= 2:
            with pytest.raises(native.W4A8Error) as e:
                call("decode")
            assert e.value.status == native.ERR_UNSUPPORTED

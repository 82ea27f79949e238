"""The MLP operators' forward calls on rows and weights of any finite size
(bounds: tests/mlp_reference.py)."""
import pytest
import torch

from tests import mlp_reference as ref
from tests.test_mlp_gpu import DT, gen, paths_for
from w4a8_quantized_gemm_channel_b200 import native

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1e35, 0.02), (1e-30, 0.02), (1e18, 1e15), (1e-10, 1e-18), (1e-25, 1e30)])
@pytest.mark.parametrize("m", [1, 12, 90])
def test_rows_and_weights_of_any_size(m, rows, cols, io):
    """Finite results come out finite, however the size is shared between
    rows and weights (row abs-max x weight abs-max from 1e-28 to 1e34, results
    up to 1e36), in every form."""
    k, n = 4096, 40
    rnd = gen(m)
    q, sw = ref.quantize_weights(rnd(n, k) * cols)
    wp = ref.pack(q)
    x = rnd(m, k)
    x = ((x.sign() * x.abs().clamp(min=0.5)) * rows).to(DT[io])      # every code large: sums of many units
    x[0] = x[0].abs()
    q[0] = q[0].abs()                                                # one output with all terms of one sign
    wp = ref.pack(q)
    b = rnd(n) * rows * cols
    want = ref.linear(x, q, sw, b, "none", None)
    assert float(want[0][0].abs().max()) < 1e37
    for path, got in paths_for(lambda p: native.w4a8_linear_act(x, wp, sw, bias=b, save=True, path=p)):
        for g, (w, e), what in zip(got, want, "yz"):
            ref.check(g, w, e, f"{what} {path}")
    want = ref.glu(x, q, sw, q, sw, b, None, "relu")
    for path, (_, g, u) in paths_for(lambda p: native.w4a8_glu(x, wp, sw, wp, sw, gate_bias=b, act="relu", save=True,
                                                               path=p)):
        for t, (w, e), what in zip((g, u), want[1:], "gu"):
            ref.check(t, w, e, f"{what} {path}")

"""Thin problems with long sums: few outputs, so few products in all, but
sums that one thread would walk for up to a millisecond."""
import pytest
import torch

from tests import mlp_reference as ref
from tests.test_mlp_gpu import DT, gen, rows, weights
from w4a8_quantized_gemm_channel_b200 import native

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(1, 6500, 10), (1, 65000, 1), (3, 2100, 9), (16, 4000, 1), (40, 1600, 1),
                                   (1, 129, 10), (1, 128, 10), (4, 256, 10), (4, 257, 10),
                                   (8, 512, 4), (8, 513, 4), (30, 500, 2)])
def test_long_forward_sums(io, m, k, n):
    rnd = gen(m + k)
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    x, b = rows(rnd, m, k, DT[io]), rnd(n)
    short = k <= (128 if m <= 2 else 256 if m <= 4 else 512)
    got = native.w4a8_linear_act(x, wg, sg, bias=b, act="silu", save=True)
    assert (native.last_path() == "generic") == short
    for t, (w, e), what in zip(got, ref.linear(x, qg, sg, b, "silu", None), "yz"):
        ref.check(t, w, e, what)
    got = native.w4a8_glu(x, wg, sg, wu, su, up_bias=b, save=True)
    assert (native.last_path() == "generic") == short
    for t, (w, e), what in zip(got, ref.glu(x, qg, sg, qu, su, None, b, "silu"), "hgu"):
        ref.check(t, w, e, what)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(1, 10, 6500), (1, 1, 32000), (3, 9, 2100), (16, 1, 4000), (130, 2, 200),
                                   (1, 10, 25), (1, 10, 24), (1, 10, 13), (1, 10, 12), (200, 3, 11)])
def test_long_gradient_sums(io, m, k, n):
    rnd = gen(m + n)
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    dy, g, u = rnd(m, n, std=0.01).to(DT[io]), rnd(m, n, std=2.0).to(DT[io]), rnd(m, n).to(DT[io])
    got = native.w4a8_linear_act_grad(dy, wg, sg, k, act="gelu", z=g, bias_grad=True)
    assert (native.last_path() == "generic") == (n <= 24)
    want, db = ref.linear_grad(dy, g, qg, sg, "gelu", n > 24)
    for t, w, what in zip(got, [want] + db, ("dx", "db")):
        ref.check(t, *w, what)
    got = native.w4a8_glu_grad(dy, g, u, wg, sg, wu, su, k, bias_grad=True)
    assert (native.last_path() == "generic") == (2 * n <= 24)
    want, db = ref.glu_grad(dy, g, u, qg, sg, qu, su, "silu", 2 * n > 24)
    for t, w, what in zip(got, [want] + db, ("dx", "dbg", "dbu")):
        ref.check(t, *w, what)

"""Weights that are column ranges of one wider array, the last range among
them, whose last row ends with the array."""
import pytest
import torch

from tests import mlp_reference as ref
from tests.test_mlp_gpu import DT, gen, rows, weights
from w4a8_quantized_gemm_channel_b200 import native

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(1, 192, 40), (12, 515, 70), (40, 96, 130), (150, 515, 263)])
def test_weights_side_by_side(io, m, k, n):
    rnd = gen(m + k)
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    cols = wg.shape[1]
    both = torch.full((n, 2 * cols + 16), 0x99, dtype=torch.uint8, device="cuda")
    vg, vu = both[:, 16: 16 + cols], both[:, 16 + cols:]
    vg.copy_(wg), vu.copy_(wu)
    x, dh = rows(rnd, m, k, DT[io]), rnd(m, n, std=0.01).to(DT[io])
    for path in ("auto", "tc"):
        h, g, u = native.w4a8_glu(x, vg, sg, vu, su, save=True, path=path)
        for t, (w, e), what in zip((h, g, u), ref.glu(x, qg, sg, qu, su, None, None, "silu"), "hgu"):
            ref.check(t, w, e, f"{what} {path}")
        ref.check(native.w4a8_linear_act(x, vu, su, path=path), *ref.linear(x, qu, su, None, "none", None)[0], path)
        want, _ = ref.glu_grad(dh, g, u, qg, sg, qu, su, "silu", True)
        ref.check(native.w4a8_glu_grad(dh, g, u, vg, sg, vu, su, k, path=path), *want, f"dx {path}")


def test_saved_rows_of_different_buffers():
    """One row has no stride: G and U may be rows of unlike buffers. Several
    rows need one stride."""
    rnd, k, n = gen(5), 64, 40
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    g, u = torch.zeros(3, 48, device="cuda")[:, :n], torch.zeros(3, 65, device="cuda")[:, 1:n + 1]
    x, dh = rnd(1, k), rnd(1, n)
    h, g1, u1 = native.w4a8_glu(x, wg, sg, wu, su, g=g[:1], u=u[:1])
    for t, (w, e), what in zip((h, g1, u1), ref.glu(x, qg, sg, qu, su, None, None, "silu"), "hgu"):
        ref.check(t, w, e, what)
    assert (g[1:] == 0).all() and (u[1:] == 0).all()
    want, _ = ref.glu_grad(dh, g1, u1, qg, sg, qu, su, "silu", True)
    ref.check(native.w4a8_glu_grad(dh, g1, u1, wg, sg, wu, su, k), *want, "dx")
    with pytest.raises(ValueError, match="one row stride"):
        native.w4a8_glu(rnd(3, k), wg, sg, wu, su, g=g, u=u)
    with pytest.raises(ValueError, match="one row stride"):
        native.w4a8_glu(x, wg, sg, wu, su, g=g[:1])
    with pytest.raises(ValueError, match="one row stride"):
        native.w4a8_glu_grad(rnd(3, n), g, u, wg, sg, wu, su, k)

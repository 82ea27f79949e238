"""Host-side limits of the MLP operators: sizes at the edge of what a call
takes. Every call here is refused before its made-up addresses are used (the
accepted sizes by a workspace that is too small)."""
import pytest

from tests.test_mlp_abi import ARGS, GLU, GLU_GRAD, LIN, LIN_GRAD, call
from w4a8_quantized_gemm_channel_b200 import native

lib = native.lib

TOP = (1 << 30) - 128     # the last N whose two segments, N rounded up to 128 each, fit an int


def wide(n):
    """A one-row call on n columns."""
    return dict(M=1, N=n, ldy=n, lddy=n, ldz=n, ldh=n, lddh=n, ldgu=n, wsb=10)


@pytest.mark.parametrize("name,n,want", [
    (GLU_GRAD, TOP, native.ERR_WORKSPACE), (GLU_GRAD, TOP + 1, native.ERR_INVALID_ARG),
    (GLU_GRAD, (1 << 30) - 1, native.ERR_INVALID_ARG),
    # one segment, and the forward calls, whose rows are K wide
    (LIN_GRAD, (1 << 30) - 1, native.ERR_WORKSPACE), (LIN, (1 << 30) - 1, native.ERR_WORKSPACE),
    (GLU, (1 << 30) - 1, native.ERR_WORKSPACE)])
def test_widest_gradient_rows(name, n, want):
    kw = {k: v for k, v in wide(n).items() if k in ARGS[name]}
    assert call(name, **kw) == want


def test_widest_gradient_rows_workspace():
    for flags in (native.IO_F32, native.IO_BF16):
        size = lib.w4a8_grad_workspace_size(1, 64, TOP, 2, flags)
        planes = 1 if flags else 2
        assert size >= planes * 2 * TOP * 2                   # FP16 rows of two segments
        assert lib.w4a8_grad_workspace_size(1, 64, TOP + 1, 2, flags) == 0
        assert lib.w4a8_grad_workspace_size(1, 64, TOP + 1, 1, flags) >= planes * TOP * 2


@pytest.mark.parametrize("m,k,n,flags", [
    (1 << 30, 64, 8, 0), (1, 64, 1 << 30, 0), (1, 64, 2 ** 31 - 1, 0), (2 ** 31 - 1, 64, 8, 0),
    (1, 64, 8, native.RELU), (1, 64, 8, native.OUT_BF16), (1, 64, 8, 0x200)])
def test_rejected_sizes_and_flags_need_no_workspace(m, k, n, flags):
    for projections in (1, 2):
        assert lib.w4a8_act_workspace_size(m, k, n, projections, flags) == 0
        assert lib.w4a8_grad_workspace_size(m, k, n, projections, flags) == 0

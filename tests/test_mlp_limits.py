"""Host-side limits of the MLP operators: sizes at the edge of what a call
takes. Every call here is refused before its made-up addresses are used (the
accepted sizes by a workspace that is too small)."""
import pytest
import torch

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


class Rows:
    """What the binding asks of a row tensor, without its memory."""
    is_cuda = True

    def __init__(self, shape, strides, dtype=torch.float32):
        self.shape, self.strides, self.dtype = torch.Size(shape), strides, dtype

    def dim(self):
        return 2

    def stride(self):
        return self.strides

    def get_device(self):
        return 0


def test_binding_passes_no_size_that_an_int_cuts_off():
    big = 2 ** 32 + 8            # an int holds its low half, 8
    assert native._rows_in(Rows((3, 8), (2 ** 31 - 1, 1)), "X") == (3, 8, 2 ** 31 - 1, 0)
    for t in (Rows((3, 8), (big, 1)), Rows((big, 8), (8, 1)), Rows((3, big), (big, 1)), Rows((1, big), (big, 1))):
        with pytest.raises(ValueError, match="fit an int"):
            native._rows_in(t, "X")
    assert native._rows_in(Rows((1, 8), (big, 1)), "X") == (1, 8, 8, 0)      # one row: its stride means nothing
    for t, k in ((Rows((big, 16), (16, 1), torch.uint8), 8), (Rows((4, big), (big, 1), torch.uint8), 8),
                 (Rows((4, big), (big, 1), torch.uint8), big)):
        with pytest.raises(ValueError, match="fit an int"):
            native._codes(t, "wp", k, 0)


def test_single_saved_rows_have_no_stride():
    a, b = torch.zeros(2, 48)[:, :40], torch.zeros(2, 64)[:, :40]
    assert native._saved(a[:1], b[:1], a, -1, 1, 40) == 40
    assert native._saved(a, a, a, -1, 2, 40) == 48 and native._saved(None, None, a, -1, 2, 40) == 0
    for g, u, m in ((a, b, 2), (a[:1], None, 1), (None, b, 2), (a[:0], None, 0)):
        with pytest.raises(ValueError, match="one row stride"):
            native._saved(g, u, a, -1, m, 40)

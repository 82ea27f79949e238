"""Host-side checks of the MLP operators: bad arguments are refused before any
device work, the size queries hold, and the reference's derivatives are those
of its functions."""
import pytest
import torch

from tests import mlp_reference as ref
from w4a8_quantized_gemm_channel_b200 import native

lib = native.lib


ARGS = {
    "w4a8_linear_act": dict(X=16, M=4, K=64, ldx=64, Wp=4096, ldp=32, sw=8192, N=8, bias=None, act=0, R=None, ldr=0,
                            flags=0, Y=12288, ldy=8, Z=None, ldz=0, ws=16384, wsb=1 << 20),
    "w4a8_glu": dict(X=16, M=4, K=64, ldx=64, Wg=4096, sg=8192, Wu=4608, su=8704, ldp=32, N=8, bg=None, bu=None,
                     act=2, flags=0, H=12288, ldh=8, G=None, U=None, ldgu=0, ws=16384, wsb=1 << 20),
    "w4a8_linear_act_grad": dict(dY=16, M=4, N=8, lddy=8, Z=1024, ldz=8, Wp=4096, ldp=32, sw=8192, K=64, act=2,
                                 flags=0, dX=12288, lddx=64, db=None, ws=16384, wsb=1 << 20),
    "w4a8_glu_grad": dict(dH=16, M=4, N=8, lddh=8, G=1024, U=2048, ldgu=8, Wg=4096, sg=8192, Wu=4608, su=8704,
                          ldp=32, K=64, act=2, flags=0, dX=12288, lddx=64, dbg=None, dbu=None, ws=16384, wsb=1 << 20),
}


def call(name, **kw):
    """The C call on made-up addresses; every case here must be refused before
    they are used. Strides that the call does not have are dropped."""
    a = dict(ARGS[name])
    a.update({k: v for k, v in kw.items() if k in a or not k.startswith("ld")})
    assert len(a) == len(ARGS[name]), kw
    return getattr(lib, name)(*a.values(), None)


LIN, GLU, LIN_GRAD, GLU_GRAD = ARGS
COMMON = [(dict(K=0), 1), (dict(N=0), 1), (dict(M=-1), 1), (dict(K=131073, ldx=1 << 20, lddx=1 << 20, ldp=1 << 17), 1),
          (dict(N=1 << 30, ldy=1 << 30, ldh=1 << 30, lddy=1 << 30, lddh=1 << 30), 1), (dict(M=1 << 30), 1),
          (dict(ldp=16), 1), (dict(ldp=40), 1), (dict(act=5), 1), (dict(act=-1), 1),
          (dict(flags=0x01), 1), (dict(flags=0x02), 1), (dict(flags=0x04), 1), (dict(flags=0x200), 1),
          (dict(ws=None), 3), (dict(wsb=10), 3), (dict(ws=16392), 3)]


@pytest.mark.parametrize("name", ARGS)
@pytest.mark.parametrize("kw,want", COMMON)
def test_sizes_flags_and_workspace(name, kw, want):
    assert call(name, **kw) == want


@pytest.mark.parametrize("name,kw", [
    (LIN, dict(X=None)), (LIN, dict(Y=None)), (LIN, dict(Wp=None)), (LIN, dict(sw=None)),
    (LIN, dict(Wp=4104)), (LIN, dict(sw=8193)), (LIN, dict(bias=2)), (LIN, dict(ldx=63)),
    (LIN, dict(ldy=7)), (LIN, dict(R=64, ldr=7)), (LIN, dict(R=66, ldr=8)), (LIN, dict(Z=64, ldz=7)),
    (LIN, dict(X=17, flags=0x100)), (LIN, dict(X=18)),
    (GLU, dict(X=None)), (GLU, dict(H=None)), (GLU, dict(Wg=None)), (GLU, dict(Wu=None)), (GLU, dict(su=None)),
    (GLU, dict(Wu=4616)), (GLU, dict(bu=2)), (GLU, dict(G=64, ldgu=8)), (GLU, dict(U=64, ldgu=8)),
    (GLU, dict(G=64, U=1024, ldgu=7)), (GLU, dict(ldh=7)), (GLU, dict(G=65, U=1024, ldgu=8, flags=0x100)),
    (LIN_GRAD, dict(dY=None)), (LIN_GRAD, dict(Z=None)), (LIN_GRAD, dict(dX=None)),
    (LIN_GRAD, dict(lddy=7)), (LIN_GRAD, dict(ldz=7)), (LIN_GRAD, dict(lddx=63)),
    (LIN_GRAD, dict(db=2)), (LIN_GRAD, dict(sw=None)),
    (GLU_GRAD, dict(dH=None)), (GLU_GRAD, dict(G=None)), (GLU_GRAD, dict(U=None)), (GLU_GRAD, dict(ldgu=7)),
    (GLU_GRAD, dict(dX=None)), (GLU_GRAD, dict(dbu=2)), (GLU_GRAD, dict(su=None)),
])
def test_pointers_and_strides(name, kw):
    assert call(name, **kw) == native.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ARGS)
def test_no_rows_and_no_device(name):
    assert call(name, M=0, ws=None, wsb=0) == native.OK
    if not torch.cuda.is_available():
        assert call(name) == native.ERR_UNSUPPORTED


def test_workspace_sizes():
    for bad in ((-1, 8, 8, 1), (1, 0, 8, 1), (1, 8, 0, 1), (1, 8, 8, 0), (1, 8, 8, 3), (1, 131073, 8, 1)):
        assert lib.w4a8_act_workspace_size(*bad, 0) == 0 and lib.w4a8_grad_workspace_size(*bad, 0) == 0
    # INT8 rows and scales; FP16 rows (two planes for float32), powers, partial bias sums
    assert native.act_workspace_size(16, 4096, 8) >= 16 * 4096 + 16 * 4
    n = native.grad_workspace_size(300, 64, 100, 2, torch.bfloat16)
    assert n >= 2 * 300 * 2 * 100 + 4 * 300 + 2 * 2 * 4 * 100
    assert native.grad_workspace_size(300, 64, 100, 2, torch.float32) >= n + 2 * 300 * 2 * 100


def test_binding_constants_match_the_header():
    from tests.test_abi import header_defines
    d = header_defines()
    for name in ("ACT_NONE", "ACT_RELU", "ACT_SILU", "ACT_GELU", "ACT_GELU_TANH", "IO_F32", "IO_BF16", "ACT_MAX_K"):
        assert getattr(native, name) == d["W4A8_" + name], name


def test_binding_refuses_mismatched_tensors():
    x, wp, sw = torch.zeros(2, 8), torch.zeros(4, 16, dtype=torch.uint8), torch.ones(4)
    ok = dict(x=x, wp=wp, sw=sw)
    for kw in (dict(x=x.half()), dict(x=x.T), dict(sw=sw.double()), dict(sw=torch.ones(5)),
               dict(wp=wp.to(torch.int8)), dict(wp=wp[:, :0]), dict(bias=torch.ones(3)),
               dict(residual=torch.zeros(2, 5)), dict(residual=torch.zeros(2, 4, dtype=torch.bfloat16)),
               dict(y=torch.zeros(4, 2).T), dict(z=torch.zeros(3, 4))):
        with pytest.raises(ValueError):
            native.w4a8_linear_act(**dict(ok, **kw))
    with pytest.raises(ValueError):
        native.w4a8_linear_act(**ok, act="swish")
    with pytest.raises(ValueError):      # the projections must agree
        native.w4a8_glu(x, wp, sw, torch.zeros(5, 16, dtype=torch.uint8), sw)
    with pytest.raises(ValueError):      # G without U
        native.w4a8_glu(x, wp, sw, wp, sw, g=torch.zeros(2, 4))
    with pytest.raises(ValueError):      # dY of another width
        native.w4a8_linear_act_grad(torch.zeros(2, 5), wp, sw, 8)
    with pytest.raises(ValueError):
        native.w4a8_glu_grad(torch.zeros(2, 4), torch.zeros(2, 4), torch.zeros(1, 4), wp, sw, wp, sw, 8)


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_reference_gradients_are_differences(name):
    """The formulas of the gradient calls against central differences of the
    float64 function on unquantized rows (the straight-through function)."""
    gen = torch.Generator().manual_seed(5)
    m, k, n = 3, 7, 5
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    (qg, sg), (qu, su) = (ref.quantize_weights(rnd(n, k).float()) for _ in range(2))
    x, dh, bg, bu = rnd(m, k), rnd(m, n), rnd(n), rnd(n)
    W = lambda q, s: (q.double() / s.double()[:, None]).T

    def f_glu(x, bg, bu):
        return (ref.act(name, x @ W(qg, sg) + bg)[0] * (x @ W(qu, su) + bu) * dh).sum()

    def f_lin(x, bg):
        return (ref.act(name, x @ W(qg, sg) + bg)[0] * dh).sum()

    def diff(f, args, i, h=1e-6):
        out = torch.zeros_like(args[i])
        for j in range(out.numel()):
            e = torch.zeros_like(args[i]).view(-1)
            e[j] = h
            e = e.view_as(args[i])
            hi, lo = list(args), list(args)
            hi[i], lo[i] = args[i] + e, args[i] - e
            out.view(-1)[j] = (f(*hi) - f(*lo)) / (2 * h)
        return out

    g, u = x @ W(qg, sg) + bg, x @ W(qu, su) + bu
    a, da = ref.act(name, g)
    segs = [(dh * u * da, 0 * g, qg, sg), (dh * a, 0 * g, qu, su)]
    (dx, _), db = ref.grad(torch.float32, segs, False)
    for want, got in zip((dx, db[0][0], db[1][0]), (diff(f_glu, (x, bg, bu), i) for i in range(3))):
        assert torch.allclose(got, want, rtol=1e-6, atol=1e-7)
    (dx, _), db = ref.grad(torch.float32, [(dh * da, 0 * g, qg, sg)], False)
    for want, got in zip((dx, db[0][0]), (diff(f_lin, (x, bg), i) for i in range(2))):
        assert torch.allclose(got, want, rtol=1e-6, atol=1e-7)

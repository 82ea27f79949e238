"""The activations and derivatives of the MLP kernels, value by value.

A zero row makes the pre-activation the bias itself, and one row of gradients
makes the bias gradient the derivative itself, so the calls give act(z),
act'(z) and the backward pass's own act(z) for any float32 z. (mlp_reference
derives its bounds for activations from other functions; the first test here
shows that they hold for these.)

Bounds from the kernel's arithmetic (U = 2^-24, first order). ex2.approx: 4 U
relative; rcp.approx: 2 U; every other float32 operation and constant: U.
  exponent  an argument A (in nats) that is off by r U of itself moves exp by
            r |A| U: r = 2 for SiLU (product, constant), 2.5 for GELU's z^2 / 2
            (square, product, half the constant's U), 4 for tanh GELU's 2t.
  logistic  s = 1 / (1 + e): e's error weighed by 1 - s, the sum and the
            reciprocal, E (1 - s) + 3 with E = r |A| + 4; c = e s: E + that + 1.
  normal    the tail q = e g: E of e, g's polynomial 7, its argument t (fma,
            reciprocal: 3 U, and g moves by at most 2.7 of t's), 1 product:
            E + 17. Phi = 1 - q for z >= 0: that times q, and U.
Results below 2^-110 may be flushed: the exponential's and the reciprocal's
smallest values, times |z|.
"""
import math

import pytest
import torch

from tests import mlp_reference as ref

U = ref.U
FLUSH = 2.0 ** -110


def bounds(name, z):
    """(bound of act, bound of act') at float64 z."""
    a, d = ref.act(name, z)
    if name in ("none", "relu"):
        return 0 * z, 0 * z
    if name == "gelu":
        q = 0.5 * torch.special.erfc(z.abs() / math.sqrt(2.0))
        dens = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        ee = 1.25 * z * z + 4
        p = torch.where(z < 0, q * (ee + 17), q * (ee + 17) + 1)          # in U
        return U * (z.abs() * p + 1.01 * a.abs()) + FLUSH, U * (p + z.abs() * dens * (ee + 4) + 1.01 * d.abs()) + FLUSH
    if name == "silu":
        arg, r, k = z, 2, 0 * z + 1
    else:
        c = math.sqrt(2 / math.pi)
        arg, r, k = 2 * c * (z + 0.044715 * z ** 3), 4, 2 * c * (1 + 3 * 0.044715 * z * z)
    s, co = torch.sigmoid(arg), torch.sigmoid(-arg)
    ee = r * arg.abs() + 4
    es = ee * co + 3
    ec = ee + es + 1
    val = U * a.abs() * (es + 1.01) + FLUSH
    if name == "silu":   # s (1 + z c)
        return val, U * (s * (z * co).abs() * (ec + 1) + s * (1 + z * co).abs() * (es + 2.01)) + FLUSH
    # s + (z s c) k: two products and k's four operations
    return val, U * ((a * co * k).abs() * (es + ec + 7) + s * es + 1.01 * d.abs()) + FLUSH


def values(device="cpu"):
    g = torch.Generator().manual_seed(1)
    mag = torch.logspace(-30, math.log10(13.0), 2000)
    z = torch.cat([torch.linspace(-13.0, 13.0, 20001), mag, -mag, torch.randn(20000, generator=g) * 3,
                   torch.tensor([0.0, -0.0, 30.0, -30.0, 80.0, -80.0])])
    return z.float().to(device)


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_derived_bounds_lie_within_the_reference_s(name):
    """What mlp_reference allows every activation (24 U of the value and 2 U)
    and derivative (32 U) covers the kernel's arithmetic."""
    z = values().double()
    ba, bd = bounds(name, z)
    assert (ba <= 24 * U * ref.act(name, z)[0].abs() + 2 * U).all()
    assert (bd <= 32 * U).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("path", ["generic", "decode", "tc"])
def test_values_and_tails(name, path):
    from w4a8_quantized_gemm_channel_b200 import native
    z = values("cuda")
    n = z.numel()
    zd = z.double()
    a, d = ref.act(name, zd)
    ba, bd = bounds(name, zd)
    wp, sw = torch.zeros((n, 16), dtype=torch.uint8, device="cuda"), torch.ones(n, device="cuda")
    zero = torch.zeros((1, 8), device="cuda")
    y, saved = native.w4a8_linear_act(zero, wp, sw, bias=z, act=name, save=True, path=path)
    assert torch.equal(saved[0], z)
    ref.check(y[0], a, ba, "act")
    one = torch.ones(n, device="cuda")
    h = native.w4a8_glu(zero, wp, sw, wp, sw, gate_bias=z, up_bias=one, act=name, path=path)
    ref.check(h[0], a, ba, "gated act")
    if path == "decode":
        return
    rows = z[None].contiguous()
    _, db = native.w4a8_linear_act_grad(one[None], wp, sw, 8, act=name, z=rows, bias_grad=True, path=path)
    ref.check(db, d, bd, "derivative")
    _, dg, du = native.w4a8_glu_grad(one[None], rows, one[None], wp, sw, wp, sw, 8, act=name, bias_grad=True, path=path)
    ref.check(dg, d, bd, "gate derivative")
    ref.check(du, a, ba, "backward act")

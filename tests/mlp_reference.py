"""float64 statements of the MLP operators and the error bounds of a correct
kernel, for the tests. U = 2^-24 is the relative error of one float32 rounding.

The integers (row codes, weight codes) are decided in float32 by the layer's
definition, so the reference decides them in float32 too; everything after is
float64.

Forward bound. acc is exact; float(acc), 1/sx, 1/sw and the two products round
once each: 5 U |p| for p = acc / (sx sw), and one more U |z| for the bias. The
activations have slopes of at most 1.13 and are evaluated from expf (2 ulp),
a fast division (2 ulp) and a few products, or normcdff (5 ulp): at most 24 U
of the value; the tanh form's argument 2t rounds by at most 4 U of itself,
which moves z s(2t) by |z| |2t| s (1 - s) 4 U <= 2 U (the product is below
0.3 for every z). Sums and products after that add one U each, and a
bfloat16 output half a step, 2^-8 of its value.

Gradient bound. The derivatives lie in [-0.13, 1.13] and are sums of products
of the same ingredients: at most 32 U absolute. Each v = dz / sw is held as
fp16(v 2^e), 2^-11 of v (float32 rows: a second term, 2^-22), plus 2^-39 of the
row's largest |v| where FP16 is subnormal; the codes are exact. The sum adds,
per accumulation step, 2^-23 of the sum of |v q| (a truncating adder): N
steps for one product at a time, (N / 16) per plane on the tensor cores, 16
products a step, and 16 more to join partial sums.
"""
import math

import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def quantize_weights(w):
    """W [N][K] float32 -> codes int8 [N][K], scales float32 [N]."""
    amax = w.abs().amax(dim=1)
    sw = torch.where(amax > 0, 7.0 / amax, torch.ones_like(amax))
    return torch.round(w * sw[:, None]).clamp(-8, 7).to(torch.int8), sw


def pack(q, ldp=None):
    n, k = q.shape
    need = ((k + 1) // 2 + 15) // 16 * 16
    ldp = need if ldp is None else ldp
    full = torch.zeros((n, 2 * ldp), dtype=torch.uint8, device=q.device)
    full[:, :k] = q.view(torch.uint8) & 15
    return (full[:, 0::2] | (full[:, 1::2] << 4)).contiguous()


def quantize_rows(x):
    x = x.float()
    amax = x.abs().amax(dim=1)
    # a scalar over a tensor is a reciprocal and a product in torch: two roundings
    sx = torch.where(amax > 0, torch.full_like(amax, 127.0) / amax, torch.ones_like(amax))
    return torch.round(x * sx[:, None]).clamp(-127, 127).double(), sx.double()


def act(name, z):
    """Activation and derivative at float64 z."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
    r = torch.sigmoid(-2 * c * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * r * 2 * c * (1 + 3 * 0.044715 * z * z)


def project(x, q, sw, bias):
    """(z, bound of a kernel's float32 z before any output rounding)."""
    xq, sx = quantize_rows(x)
    p = (xq @ q.double().T) / sx[:, None] / sw.double()
    z = p if bias is None else p + bias.double()
    return z, 5 * U * p.abs() + U * z.abs()


def linear(x, q, sw, bias, name, residual):
    """[(y, bound), (z, bound)] with the output rounding of x's dtype."""
    z, ez = project(x, q, sw, bias)
    a, _ = act(name, z)
    y, ey = a, 1.13 * ez + (0 if name in ("none", "relu") else 24 * U * a.abs() + 2 * U)
    if residual is not None:
        y = a + residual.double()
    h = HALF_STEP[x.dtype]
    return [(y, ey + U * y.abs() + h * y.abs()), (z, ez + h * z.abs())]


def glu(x, qg, sg, qu, su, bg, bu, name):
    g, eg = project(x, qg, sg, bg)
    u, eu = project(x, qu, su, bu)
    a, _ = act(name, g)
    ea = 1.13 * eg + (0 if name in ("none", "relu") else 24 * U * a.abs() + 2 * U)
    h = a * u
    s = HALF_STEP[x.dtype]
    return [(h, ea * u.abs() + (a.abs() + ea) * eu + (U + s) * h.abs()), (g, eg + s * g.abs()), (u, eu + s * u.abs())]


def grad(dtype, segments, tensor_cores):
    """segments: [(dz, error bound of a float32 dz, q, sw)]; returns
    (dx, bound), [(dbias, bound)]."""
    dx, spread, verr, steps = 0, 0, 0, 16
    planes = 2 if dtype == torch.float32 else 1
    top = torch.stack([(dz / sw.double()).abs().amax(dim=1) for dz, _, _, sw in segments]).amax(dim=0)
    for dz, edz, q, sw in segments:
        v, ev, qd = dz / sw.double(), edz / sw.double(), q.double()
        dx = dx + v @ qd
        spread = spread + v.abs() @ qd.abs()
        held = (2.0 ** -22 if planes == 2 else 2.0 ** -11) * v.abs() + 2.0 ** -39 * top[:, None]
        verr = verr + (ev + U * v.abs() + held) @ qd.abs()
        steps += -(-v.shape[1] // 16) * planes if tensor_cores else v.shape[1]
    bound = verr + steps * 2.0 ** -23 * spread + (U + HALF_STEP[dtype]) * dx.abs()
    m = segments[0][0].shape[0]
    db = [(dz.sum(0), edz.sum(0) + (m + 16) * U * dz.abs().sum(0)) for dz, edz, _, _ in segments]
    return (dx, bound), db


def linear_grad(dy, z, q, sw, name, tensor_cores):
    d = dy.double()
    if name == "none":
        dz, e = d, 0 * d
    else:
        dz = d * act(name, z.double())[1]
        e = d.abs() * 32 * U + U * dz.abs()
    return grad(dy.dtype, [(dz, e, q, sw)], tensor_cores)


def glu_grad(dh, g, u, qg, sg, qu, su, name, tensor_cores):
    a, da = act(name, g.double())
    d, ud = dh.double(), u.double()
    dg, du = d * ud * da, d * a
    eg = (d * ud).abs() * 32 * U + 2 * U * dg.abs()
    eu = d.abs() * (24 * U * a.abs() + 2 * U) + U * du.abs()
    return grad(dh.dtype, [(dg, eg, qg, sg), (du, eu, qu, su)], tensor_cores)


def check(got, want, bound, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: non-finite output"
    bad = err > bound
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outputs off, first at {i}: got "
                             f"{float(got[i])!r}, want {float(want[i])!r}, bound {float(bound[i])!r}")

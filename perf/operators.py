"""Measured cases of the MLP operators: the W4A8 product with bias, activation
and residual in its epilogue, the gated feed-forward product, and the input
gradients of both.

With `own` false `run` computes an operator in its plain form (elementary torch
operations in float32 on the unpacked weights, rounded once at the end); with
`own` true it makes the library's calls. `exact` gives the operator's
definition in float64.

Definitions (T = the case's "io" type: x, residual, outputs, gradients):
  rows     sx = 127 / max|x| (1 for a zero row), xq = clamp(rne(x * sx)), both
           decided in float32 as the layer defines them;
  weights  w = q / sw, codes q in [-8, 7], two per byte along K;
  linear   z = xq . q / (sx sw) + bias, y = act(z) + residual;
  linear_grad  dz = dy act'(z), dx = dz . w^T, dbias = sum over rows of dz;
  glu      g, u = the two projections, h = act(g) u;
  glu_grad dg = dh u act'(g), du = dh act(g), dx = dg . wg^T + du . wu^T.
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16}
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------- cases ---

def _case(name, op, io, m, k, n, act, bias=False, residual=False, save=False):
    return {"name": name, "op": op, "io": io, "m": m, "k": k, "n": n, "act": act, "bias": bias,
            "residual": residual, "save": save}


def listed():
    return [
        # the smallest call: the first layer of the two-layer model the tests and the smoke run use
        _case("linear_tiny", "linear", "f32", 32, 10, 32, "relu", bias=True),
        # down projection of one token with the residual stream added, decode of a 4096 / 11008 block
        _case("linear_decode", "linear", "bf16", 1, 11008, 4096, "none", residual=True),
        # up projection of an ungated block of the 1152 / 6912 stack, a ragged batch, float32 rows, all of the epilogue
        _case("linear_ragged", "linear", "f32", 333, 1151, 6913, "gelu", bias=True, residual=True),
        # down projection of a prompt of 2048 tokens with its residual
        _case("linear_prompt", "linear", "bf16", 2048, 11008, 4096, "none", residual=True),
        # gate and up projections of one token
        _case("glu_decode", "glu", "bf16", 1, 4096, 11008, "silu"),
        # a small decode batch through the 1152 / 6912 stack
        _case("glu_batch", "glu", "bf16", 16, 1152, 6912, "gelu_tanh"),
        # forward of a training step: pre-activations saved for the backward pass, biases, float32
        _case("glu_train", "glu", "f32", 1000, 1152, 6912, "gelu_tanh", bias=True, save=True),
        # a prompt through the gate and up projections of an 8192 / 28672 block: the largest
        _case("glu_prompt", "glu", "bf16", 2048, 8192, 28672, "silu"),
        # gradient below a short float32 batch, odd sizes, with the bias gradient
        _case("linear_grad_ragged", "linear_grad", "f32", 129, 1151, 1001, "gelu_tanh", bias=True),
        # gradient through the down projection of a 2048-token training batch
        _case("linear_grad_train", "linear_grad", "bf16", 2048, 11008, 4096, "none"),
        # gradient through the gated pair, a short batch of the 1152 / 6912 stack in float32
        _case("glu_grad_short", "glu_grad", "f32", 200, 1152, 6912, "gelu_tanh", bias=True),
        # gradient through the gated pair, 2048 training tokens
        _case("glu_grad_train", "glu_grad", "bf16", 2048, 4096, 11008, "silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "glu", "linear_grad", "glu_grad"])
    k, n = _log(rng, 10, 11008), _log(rng, 10, 28672)
    m = _log(rng, 1, 2048)
    if rng.random() < 0.5:  # half of the calls have the aligned sizes of a model
        k, n = max(16, k // 16 * 16), max(16, n // 16 * 16)
    io = rng.choice(["f32", "bf16"])
    grad = op.endswith("_grad")
    return {"op": op, "io": io, "m": m, "k": k, "n": n, "act": rng.choice(_ACTS), "bias": rng.random() < 0.5,
            "residual": op == "linear" and rng.random() < 0.5, "save": not grad and rng.random() < 0.3}


def work(case):
    m, k, n, e = case["m"], case["k"], case["n"], _T[case["io"]].itemsize
    two = 2 if case["op"].startswith("glu") else 1
    grad = case["op"].endswith("_grad")
    weights = two * (n * ((k + 1) // 2) + 4 * n)
    extra = two * 4 * n if case["bias"] else 0            # biases read, or their gradients written
    if grad:
        saved = 2 if two == 2 else (0 if case["act"] == "none" else 1)
        rows = m * k * e + (1 + saved) * m * n * e
    else:
        outs = 1 + (two if case["save"] else 0) + (1 if case["residual"] else 0)
        rows = m * k * e + outs * m * n * e
    return {"bytes": weights + extra + rows, "flops": 2 * two * m * n * k}


# ------------------------------------------------------------------ inputs ---

def _inputs(case, seed):
    """Everything random, from the seed alone: weight codes and scales as the
    layer's weight quantization gives them, rows with a few large channels."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    m, k, n, t = case["m"], case["k"], case["n"], _T[case["io"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    d = {}
    for name in ("g", "u") if case["op"].startswith("glu") else ("w",):
        w = normal(n, k, std=0.02)                        # [N][K]: the layer's kernel, transposed
        amax = w.abs().amax(dim=1)
        sw = torch.where(amax > 0, 7.0 / amax, torch.ones_like(amax))
        d["q" + name] = torch.round(w * sw[:, None]).clamp_(-8, 7).to(torch.int8)
        d["s" + name] = sw
        del w
        if case["bias"] and not case["op"].endswith("_grad"):
            d["b" + name] = normal(n, std=0.1)
    if case["op"].endswith("_grad"):
        d["dy"] = normal(m, n, std=0.01).to(t)
        # the saved pre-activations (a plain product without activation needs none)
        for name in ("zg", "zu") if case["op"] == "glu_grad" else ("z",) if case["act"] != "none" else ():
            d[name] = normal(m, n, std=1.5).to(t)
        return d
    x = normal(m, k)
    big = torch.randperm(k, generator=gen, device=dev)[: max(1, round(0.005 * k))]
    x[:, big] *= 20.0                                     # outlier channels, as activations have them
    d["x"] = x.to(t)
    if case["residual"]:
        d["r"] = normal(m, n, std=2.0).to(t)
    return d


def _pack(q):
    """Codes [N][K] -> bytes [N][ldp]: even k in the low nibble, rows padded to 16 bytes."""
    n, k = q.shape
    ldp = ((k + 1) // 2 + 15) // 16 * 16
    full = torch.zeros((n, 2 * ldp), dtype=torch.uint8, device=q.device)
    full[:, :k] = q.view(torch.uint8) & 15
    return full[:, 0::2] | (full[:, 1::2] << 4)


def prepare(case, seed):
    d = _inputs(case, seed)
    state = {"case": case}
    for name, v in d.items():
        if name[0] == "q":
            state["p" + name[1:]] = _pack(v)
        else:
            state[name] = v
    if own:
        from w4a8_quantized_gemm_channel_b200 import native
        m, k, n = case["m"], case["k"], case["n"]
        size_of = native.grad_workspace_size if case["op"].endswith("_grad") else native.act_workspace_size
        size = size_of(m, k, n, projections=2 if case["op"].startswith("glu") else 1, dtype=_T[case["io"]])
        state["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return state


# -------------------------------------------------------------- plain form ---

def _unpack(p, k):
    """Bytes [N][ldp] -> float32 codes [N][K]."""
    lo = ((p & 15) ^ 8).to(torch.int8) - 8
    hi = ((p >> 4) ^ 8).to(torch.int8) - 8
    return torch.stack((lo, hi), dim=2).reshape(p.shape[0], -1)[:, :k].float()


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _act(act, z):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * _sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    t = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    return z * _sigmoid(2.0 * t)


def _act_grad(act, z):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = _sigmoid(z)
        return s * (1.0 + z * _sigmoid(-z))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = c * (z + 0.044715 * z * z * z)
    s = _sigmoid(2.0 * t)
    return s + z * s * _sigmoid(-2.0 * t) * 2.0 * c * (1.0 + 3.0 * 0.044715 * z * z)


def _plain_project(xq, sx, p, sw, k, bias):
    # integers up to 127 * 8 * k: float32 holds every partial sum exactly to k = 16512
    acc = xq @ _unpack(p, k).T
    z = acc / (sx * sw)
    return z if bias is None else z + bias


def _run_plain(s):
    c = s["case"]
    t, k, act = _T[c["io"]], c["k"], c["act"]
    if c["op"].endswith("_grad"):
        dy = s["dy"].float()
        if c["op"] == "glu_grad":
            g, u = s["zg"].float(), s["zu"].float()
            parts = [(dy * u * _act_grad(act, g), "g"), (dy * _act(act, g), "u")]
        else:
            parts = [(dy if act == "none" else dy * _act_grad(act, s["z"].float()), "w")]
        dx = sum((dz / s["s" + n]) @ _unpack(s["p" + n], k) for dz, n in parts)
        out = [dx.to(t)]
        if c["bias"]:
            out += [dz.double().sum(dim=0).float() for dz, _ in parts]
        return out
    x = s["x"].float()
    amax = x.abs().amax(dim=1, keepdim=True)
    # one rounded division (a scalar over a tensor would be a reciprocal and a product)
    sx = torch.where(amax > 0, torch.full_like(amax, 127.0) / amax, torch.ones_like(amax))
    xq = torch.round(x * sx).clamp(-127, 127)
    if c["op"] == "linear":
        z = _plain_project(xq, sx, s["pw"], s["sw"], k, s.get("bw"))
        y = _act(act, z)
        if c["residual"]:
            y = y + s["r"].float()
        return [y.to(t)] + ([z.to(t)] if c["save"] else [])
    g = _plain_project(xq, sx, s["pg"], s["sg"], k, s.get("bg"))
    u = _plain_project(xq, sx, s["pu"], s["su"], k, s.get("bu"))
    return [(_act(act, g) * u).to(t)] + ([g.to(t), u.to(t)] if c["save"] else [])


# ------------------------------------------------------- the library's calls ---

def _run_own(s):
    from w4a8_quantized_gemm_channel_b200 import native
    c = s["case"]
    # the weights are frozen and settled, as in a program that serves or trains on top of them
    kw = {"act": c["act"], "workspace": s["ws"], "static_weights": True}
    if c["op"] == "linear":
        out = native.w4a8_linear_act(s["x"], s["pw"], s["sw"], bias=s.get("bw"), residual=s.get("r"),
                                     save=c["save"], **kw)
    elif c["op"] == "glu":
        out = native.w4a8_glu(s["x"], s["pg"], s["sg"], s["pu"], s["su"], gate_bias=s.get("bg"),
                              up_bias=s.get("bu"), save=c["save"], **kw)
    elif c["op"] == "linear_grad":
        out = native.w4a8_linear_act_grad(s["dy"], s["pw"], s["sw"], c["k"], z=s.get("z"),
                                          bias_grad=c["bias"], **kw)
    else:
        out = native.w4a8_glu_grad(s["dy"], s["zg"], s["zu"], s["pg"], s["sg"], s["pu"], s["su"], c["k"],
                                   bias_grad=c["bias"], **kw)
    return list(out) if isinstance(out, tuple) else [out]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------- in 64 bits ---

def _cdf(v):
    return torch.special.ndtr(v)


def _exact_act(act, z):
    """act(z) and its derivative, float64, from their textbook forms."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        pos = (z > 0).double()
        return z * pos, pos
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return z * _cdf(z), _cdf(z) + z * torch.exp(-z * z / 2.0) / (2.0 * math.pi) ** 0.5
    r = (2.0 / math.pi) ** 0.5
    th = torch.tanh(r * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * r * (1.0 + 0.134145 * z * z)


def exact(case, seed):
    d = _inputs(case, seed)
    act, t = case["act"], case["op"]
    if t == "linear_grad":
        dz = d["dy"].double()
        if act != "none":
            dz = dz * _exact_act(act, d["z"].double())[1]
        dx = (dz / d["sw"].double()) @ d["qw"].double()
        return [dx] + ([dz.sum(0)] if case["bias"] else [])
    if t == "glu_grad":
        a, da = _exact_act(act, d["zg"].double())
        dy = d["dy"].double()
        dg, du = dy * d["zu"].double() * da, dy * a
        dx = (dg / d["sg"].double()) @ d["qg"].double()
        dx += (du / d["su"].double()) @ d["qu"].double()
        return [dx] + ([dg.sum(0), du.sum(0)] if case["bias"] else [])
    # the row codes are defined by float32 decisions (scale, product, rounding)
    x32 = d["x"].float()
    top = x32.abs().max(dim=1).values
    scale = torch.where(top == 0, torch.ones_like(top), torch.full_like(top, 127.0) / top)
    codes = torch.clamp(torch.round(x32 * scale.unsqueeze(1)), -127.0, 127.0).double()

    def project(n):
        z = (codes @ d["q" + n].double().t()) / scale.double().unsqueeze(1) / d["s" + n].double()
        return z + d["b" + n].double() if case["bias"] else z

    if t == "linear":
        z = project("w")
        y = _exact_act(act, z)[0]
        if case["residual"]:
            y = y + d["r"].double()
        return [y] + ([z] if case["save"] else [])
    g, u = project("g"), project("u")
    return [_exact_act(act, g)[0] * u] + ([g, u] if case["save"] else [])

"""What the MLP bindings refuse, on CUDA tensors: the unmodified call runs, and
each change alone is refused, with the message that names it."""
import pytest
import torch

from w4a8_quantized_gemm_channel_b200 import native

pytestmark = pytest.mark.gpu

M, K, N = 6, 24, 12


def f(*shape, dtype=torch.float32):
    return torch.ones(shape, dtype=dtype, device="cuda")


def codes(n=N):
    return torch.zeros((n, 16), dtype=torch.uint8, device="cuda")


CALLS = {
    "linear": (native.w4a8_linear_act, lambda: dict(x=f(M, K), wp=codes(), sw=f(N), bias=f(N), residual=f(M, N),
                                                    y=f(M, N), z=f(M, N), act="silu")),
    "glu": (native.w4a8_glu, lambda: dict(x=f(M, K), wg=codes(), sg=f(N), wu=codes(), su=f(N), gate_bias=f(N),
                                          up_bias=f(N), h=f(M, N), g=f(M, N), u=f(M, N))),
    "linear_grad": (native.w4a8_linear_act_grad, lambda: dict(dy=f(M, N), wp=codes(), sw=f(N), k=K, act="gelu",
                                                              z=f(M, N), bias_grad=True, dx=f(M, K))),
    "glu_grad": (native.w4a8_glu_grad, lambda: dict(dh=f(M, N), g=f(M, N), u=f(M, N), wg=codes(), sg=f(N), wu=codes(),
                                                    su=f(N), k=K, bias_grad=True, dx=f(M, K))),
}
half = torch.float16
bf = torch.bfloat16

ROW_NAMES = {"linear": ("x", "X", K), "glu": ("x", "X", K), "linear_grad": ("dy", "dY", N), "glu_grad": ("dh", "dH", N)}
REFUSED = [(op, {arg: change}, match)
           for op, (arg, name, cols) in ROW_NAMES.items()
           for change, match in ((lambda c=cols: f(M, c).half(), "rows must be float32 or bfloat16"),
                                 (lambda c=cols: f(M, c).cpu(), f"{name} must be a 2-D CUDA tensor"),
                                 (lambda c=cols: f(M, c, 1), f"{name} must be a 2-D CUDA tensor"),
                                 (lambda c=cols: f(c, M).T, f"{name} must have unit column stride"))]
for op, args in {"linear": ["wp"], "glu": ["wg", "wu"], "linear_grad": ["wp"], "glu_grad": ["wg", "wu"]}.items():
    for arg in args:
        REFUSED += [(op, {arg: lambda: codes().to(torch.int8)}, f"{arg} must be .*uint8"),
                    (op, {arg: lambda: codes().cpu()}, f"{arg} must be .*uint8"),
                    (op, {arg: lambda: codes()[:, :11]}, f"{arg} must be .*uint8"),       # K = 24 needs 12 bytes
                    (op, {arg: lambda: codes()[0]}, f"{arg} must be .*uint8"),
                    (op, {arg: lambda: torch.zeros((32, N), dtype=torch.uint8, device="cuda").T},
                     f"{arg} must have unit column stride")]
for op in ("glu", "glu_grad"):
    REFUSED += [(op, dict(wu=lambda: codes(N + 1)), "the same shape and row stride"),
                (op, dict(wu=lambda: torch.zeros((N, 32), dtype=torch.uint8, device="cuda")),
                 "the same shape and row stride"),
                (op, dict(u=lambda: f(M, N + 4)[:, :N]), "one row stride")]
REFUSED += [("glu", dict(u=lambda: None), "one row stride"), ("glu", dict(g=lambda: None), "one row stride"),
            ("linear_grad", dict(dy=lambda: f(M, N + 1)), f"dY must have {N} columns"),
            ("glu_grad", dict(dh=lambda: f(M, N + 1)), f"dH must have {N} columns")]
for op, args in {"linear": ["sw", "bias"], "glu": ["sg", "su", "gate_bias", "up_bias"], "linear_grad": ["sw"],
                 "glu_grad": ["sg", "su"]}.items():
    for arg in args:
        REFUSED += [(op, {arg: change}, f"{arg} must be a contiguous float32 tensor of {N} values") for change in
                    (lambda: f(N + 1), lambda: f(N - 1), lambda: f(N).double(), lambda: f(N).cpu(), lambda: f(2 * N)[::2])]
for op, args in {"linear": dict(residual=N, y=N, z=N), "glu": dict(h=N, g=N, u=N), "linear_grad": dict(z=N, dx=K),
                 "glu_grad": dict(g=N, u=N, dx=K)}.items():
    for arg, cols in args.items():
        name = arg if arg == "residual" else "dX" if arg == "dx" else arg.upper()
        REFUSED += [(op, {arg: change}, rf"{name} must be a \[{M}\]\[{cols}\] torch.float32 tensor") for change in
                    (lambda c=cols: f(M + 1, c), lambda c=cols: f(M, c + 1), lambda c=cols: f(1, c),
                     lambda c=cols: f(M, c).bfloat16(), lambda c=cols: f(M, c).cpu(), lambda c=cols: f(M * c))]
        REFUSED += [(op, {arg: lambda c=cols: f(c, M).T}, f"{name} must have unit column stride")]
for op in CALLS:
    REFUSED += [(op, dict(act=lambda: "swish"), "act one of"), (op, dict(path=lambda: "fast"), "path one of"),
                (op, dict(workspace=lambda: torch.zeros(1 << 24, dtype=torch.uint8)), "workspace must be contiguous"),
                (op, dict(workspace=lambda: torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")[::2]),
                 "workspace must be contiguous")]


@pytest.mark.parametrize("op", CALLS)
def test_the_unmodified_call_runs(op):
    fn, args = CALLS[op]
    out = fn(**args())
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in (out if isinstance(out, tuple) else (out,)))


@pytest.mark.parametrize("op,change,match", REFUSED, ids=[f"{i}-{o}-{next(iter(c))}" for i, (o, c, _) in enumerate(REFUSED)])
def test_one_change_is_refused(op, change, match):
    fn, args = CALLS[op]
    with pytest.raises(ValueError, match=match):
        fn(**dict(args(), **{k: v() for k, v in change.items()}))


@pytest.mark.parametrize("op", CALLS)
def test_library_errors(op):
    """What the library itself refuses arrives as W4A8Error with its status."""
    fn, args = CALLS[op]
    base = args()
    lead = next(iter(base))

    def status(**kw):
        with pytest.raises(native.W4A8Error) as e:
            fn(**dict(base, **kw))
        return e.value.status

    assert status(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")) == native.ERR_WORKSPACE
    assert status(workspace=torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")[8:]) == native.ERR_WORKSPACE
    rows = base[lead]
    assert status(**{lead: rows[:1].expand_as(rows)}) == native.ERR_INVALID_ARG          # rows of stride 0
    for arg in ("wp",) if "wp" in base else ("wg",):
        odd = torch.zeros((N, 24), dtype=torch.uint8, device="cuda")                      # a stride of 24 bytes
        assert status(**{a: odd for a in ("wp", "wg", "wu") if a in base}) == native.ERR_INVALID_ARG
        off = torch.zeros((N, 32), dtype=torch.uint8, device="cuda")[:, 8:24]             # rows off 16 bytes
        assert status(**{a: off for a in ("wp", "wg", "wu") if a in base}) == native.ERR_INVALID_ARG
    assert status(path="split") == native.ERR_UNSUPPORTED
    if op == "linear_grad":
        assert status(z=None) == native.ERR_INVALID_ARG


def test_a_stream_of_another_device_is_refused():
    class Elsewhere:
        device = torch.device("cuda", 7)

    for fn, args in CALLS.values():
        with pytest.raises(ValueError, match="stream is on cuda:7"):
            fn(**args(), stream=Elsewhere())

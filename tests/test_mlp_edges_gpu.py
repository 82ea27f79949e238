"""Calls of the MLP operators that the other tests do not make: more rows than
a grid holds, vectors off 16 bytes, workspaces of exactly the asked size, two
host threads, the longest sums of the gradients, the residual in place under
shared tiles, rows that are not finite beside rows that are."""
import threading

import pytest
import torch

from tests import mlp_reference as ref
from tests.test_mlp_gpu import ACTS, DT, gen, rows, weights
from w4a8_quantized_gemm_channel_b200 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    native.get_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert native.get_device_status() == 0


def all_four(x, dh, g, u, wg, sg, wu, su, k, **kw):
    return (native.w4a8_linear_act(x, wg, sg, act="gelu", residual=dh, save=True, **kw),
            native.w4a8_glu(x, wg, sg, wu, su, save=True, **kw),
            native.w4a8_linear_act_grad(dh, wg, sg, k, act="gelu", z=g, bias_grad=True, **kw),
            native.w4a8_glu_grad(dh, g, u, wg, sg, wu, su, k, bias_grad=True, **kw))


def expected(x, dh, g, u, qg, sg, qu, su, tensor_cores=True):
    lin, db = ref.linear_grad(dh, g, qg, sg, "gelu", tensor_cores)
    glu, dbs = ref.glu_grad(dh, g, u, qg, sg, qu, su, "silu", tensor_cores)
    return (ref.linear(x, qg, sg, None, "gelu", dh), ref.glu(x, qg, sg, qu, su, None, None, "silu"),
            [lin] + db, [glu] + dbs)


def check_all(got, want, what):
    for op, gs, ws in zip(("linear", "glu", "linear_grad", "glu_grad"), got, want):
        for i, (t, (w, e)) in enumerate(zip(gs, ws)):
            ref.check(t, w, e, f"{what} {op} {i}")


def problem(m, k, n, io, seed=0):
    rnd = gen(seed + m + k + n)
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    x, dh = rows(rnd, m, k, DT[io]), rnd(m, n, std=0.01).to(DT[io])
    g, u = rnd(m, n, std=2.0).to(DT[io]), rnd(m, n).to(DT[io])
    return (x, dh, g, u, wg, sg, wu, su, k), (x, dh, g, u, qg, sg, qu, su)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("path", ["generic", "tc"])
def test_more_rows_than_a_grid_has_blocks(io, path):
    """70001 rows: the row passes and the CUDA-core kernels walk on."""
    args, facts = problem(70001, 40, 72, io)
    check_all(all_four(*args, path=path), expected(*facts, path == "tc"), path)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 5, 16, 70])
def test_vectors_off_16_bytes(io, m):
    """Scales and biases that start one element into their array."""
    (x, dh, g, u, wg, sg, wu, su, k), facts = problem(m, 200, 133, io)
    off = lambda v: torch.cat([v[:1], v])[1:]
    assert off(sg).data_ptr() % 16 == 4
    check_all(all_four(x, dh, g, u, wg, off(sg), wu, off(su), k), expected(*facts), "off")
    b = torch.linspace(-1, 1, 133, device="cuda")
    same = [native.w4a8_glu(x, wg, s1, wu, s2, gate_bias=b1, up_bias=b1, save=True)
            for s1, s2, b1 in ((sg, su, b), (off(sg), off(su), off(b)))]
    assert all(torch.equal(a, c) for a, c in zip(*same))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(1, 10, 32), (1, 11008, 40), (9, 515, 260), (40, 16390, 523), (300, 1029, 77),
                                   (460, 62, 12749)])
def test_workspace_of_exactly_the_asked_size(io, m, k, n):
    """At the least alignment, with what lies before and behind left alone."""
    args, facts = problem(m, k, n, io)
    x, dh, g, u, wg, sg, wu, su, _ = args
    want = all_four(*args)
    calls = ((native.act_workspace_size, 1, lambda ws: native.w4a8_linear_act(x, wg, sg, act="gelu", residual=dh,
                                                                              save=True, workspace=ws)),
             (native.act_workspace_size, 2, lambda ws: native.w4a8_glu(x, wg, sg, wu, su, save=True, workspace=ws)),
             (native.grad_workspace_size, 1, lambda ws: native.w4a8_linear_act_grad(dh, wg, sg, k, act="gelu", z=g,
                                                                                    bias_grad=True, workspace=ws)),
             (native.grad_workspace_size, 2, lambda ws: native.w4a8_glu_grad(dh, g, u, wg, sg, wu, su, k,
                                                                             bias_grad=True, workspace=ws)))
    for (size, projections, call), out in zip(calls, want):
        need = size(m, k, n, projections, DT[io])
        for at in (16, 240, 256, 272):
            buf = torch.full((need + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
            got = call(buf[at: at + need])
            assert all(torch.equal(a, b) for a, b in zip(got, out))
            assert (buf[:at] == 0xA5).all() and (buf[at + need:] == 0xA5).all()


def test_two_host_threads():
    """Calls from two threads, each on its own stream, give the bits they give alone."""
    probs = [problem(m, 260, 700, io)[0] for m, io in ((3, "f32"), (200, "bf16"))]
    alone = [all_four(*p) for p in probs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(30):
            with torch.cuda.stream(s):
                got = all_four(*probs[i])
            s.synchronize()
            if not all(torch.equal(a, b) for x, y in zip(got, alone[i]) for a, b in zip(x, y)):
                bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(2, native.ACT_MAX_K, 9), (40, native.ACT_MAX_K - 3, 30), (3, 70, 200001),
                                   (90, 33, 150000)])
def test_longest_gradients(io, m, k, n):
    """K at its limit, and sums over many more outputs than a block holds."""
    (x, dh, g, u, wg, sg, wu, su, _), facts = problem(m, k, n, io)
    want = expected(*facts, tensor_cores=True)
    ref_bound = lambda got, ws, what: [ref.check(t, w, e, what) for t, (w, e) in zip(got, ws)]
    ref_bound(native.w4a8_linear_act_grad(dh, wg, sg, k, act="gelu", z=g, bias_grad=True, path="tc"), want[2], "linear")
    ref_bound(native.w4a8_glu_grad(dh, g, u, wg, sg, wu, su, k, bias_grad=True, path="tc"), want[3], "glu")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(40, 16390, 520), (40, 16390, 523), (67, 300, 4737), (1, 4096, 100), (16, 515, 100)])
def test_residual_in_place(io, m, k, n):
    (x, dh, _, _, wg, sg, _, _, _), (_, _, _, _, qg, _, _, _) = problem(m, k, n, io)
    want = ref.linear(x, qg, sg, None, "silu", dh)[0]
    y = dh.clone()
    for path in ("tc",) + (("auto", "decode") if m <= 16 else ()):
        y.copy_(dh)
        ref.check(native.w4a8_linear_act(x, wg, sg, act="silu", residual=y, y=y, path=path), *want, path)


@pytest.mark.parametrize("m", [2, 16, 40, 300])
def test_rows_that_are_not_finite_stay_alone(m):
    """Not-finite rows are outside the contract, but the other rows of the
    call keep their bits."""
    (x, dh, g, u, wg, sg, wu, su, k), _ = problem(m, 260, 130, "f32")
    good = all_four(x, dh, g, u, wg, sg, wu, su, k)
    x2, dh2 = x.clone(), dh.clone()
    x2[0, 3], x2[0, 9], dh2[0, 5], dh2[0, 7] = float("nan"), float("inf"), float("inf"), float("nan")
    got = all_four(x2, dh2, g, u, wg, sg, wu, su, k)
    for a, b in zip(got, good):
        for t, w in zip(a, b):
            if t.dim() == 2:
                assert torch.equal(t[1:], w[1:])
    assert not torch.isfinite(got[2][0][0]).all() and not torch.isfinite(got[3][0][0]).all()

"""The MLP operators on a B200 against their float64 statements
(tests/mlp_reference.py, which derives the bounds)."""
import pytest
import torch

from tests import mlp_reference as ref
from w4a8_quantized_gemm_channel_b200 import native

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    native.get_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert native.get_device_status() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std


def weights(rnd, n, k):
    q, sw = ref.quantize_weights(rnd(n, k, std=0.05))
    return q, sw, ref.pack(q)


def rows(rnd, m, k, dt):
    x = rnd(m, k)
    x[:, :: max(1, k // 3)] *= 20.0
    return x.to(dt)


# one row to many, K and N around the widths a kernel tiles by (8, 16, 64, 128, 256), odd ones among them
SHAPES = [(1, 1, 1), (1, 10, 32), (3, 31, 17), (5, 64, 8), (1, 2048, 264), (2, 4099, 40), (8, 1152, 333), (13, 515, 129),
          (16, 128, 256), (17, 130, 65), (40, 257, 300), (64, 1151, 128), (127, 96, 255), (129, 384, 257),
          (256, 640, 512), (300, 1029, 77)]


def paths_for(call):
    """The result of every kernel path that runs this call, AUTO first."""
    out = []
    for path in ("auto", "generic", "decode", "tc"):
        try:
            out.append((path, call(path)))
        except native.W4A8Error as e:
            assert e.status == native.ERR_UNSUPPORTED and path in ("decode", "tc")
    return out


@pytest.mark.parametrize("m,k,n", SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_act(m, k, n, io):
    rnd = gen(m * 7 + k + n)
    q, sw, wp = weights(rnd, n, k)
    x, r, b = rows(rnd, m, k, DT[io]), rnd(m, n, std=2.0).to(DT[io]), rnd(n)
    for i, act in enumerate(ACTS):
        bias, res, save = (b if i % 2 == 0 else None), (r if i % 3 != 1 else None), i % 2 == 1
        want = ref.linear(x, q, sw, bias, act, res)
        for path, got in paths_for(lambda p: native.w4a8_linear_act(x, wp, sw, bias=bias, act=act, residual=res,
                                                                    save=save, path=p)):
            got = got if save else (got,)
            for g, (w, e), what in zip(got, want, "yz"):
                ref.check(g, w, e, f"{what} {act} {path}")


@pytest.mark.parametrize("m,k,n", SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_glu(m, k, n, io):
    rnd = gen(m * 11 + k + n)
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    x, b1, b2 = rows(rnd, m, k, DT[io]), rnd(n), rnd(n)
    for i, act in enumerate(ACTS):
        bg, bu, save = (b1 if i % 2 == 0 else None), (b2 if i % 3 != 1 else None), i % 2 == 0
        want = ref.glu(x, qg, sg, qu, su, bg, bu, act)
        for path, got in paths_for(lambda p: native.w4a8_glu(x, wg, sg, wu, su, gate_bias=bg, up_bias=bu, act=act,
                                                             save=save, path=p)):
            got = got if save else (got,)
            for g, (w, e), what in zip(got, want, "hgu"):
                ref.check(g, w, e, f"{what} {act} {path}")


@pytest.mark.parametrize("m,k,n", SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_act_grad(m, k, n, io):
    rnd = gen(m * 13 + k + n)
    q, sw, wp = weights(rnd, n, k)
    dy, z = rnd(m, n, std=0.01).to(DT[io]), rnd(m, n, std=2.0).to(DT[io])
    z[:, ::5] = 0.0
    for i, act in enumerate(ACTS):
        bias = i % 2 == 0
        for path, got in paths_for(lambda p: native.w4a8_linear_act_grad(dy, wp, sw, k, act=act, z=z, bias_grad=bias,
                                                                         path=p)):
            want, db = ref.linear_grad(dy, z, q, sw, act, path == "tc")
            ref.check(got[0] if bias else got, *want, f"dx {act} {path}")
            if bias:
                ref.check(got[1], *db[0], f"db {act} {path}")


@pytest.mark.parametrize("m,k,n", SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_glu_grad(m, k, n, io):
    rnd = gen(m * 17 + k + n)
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    dh, g, u = rnd(m, n, std=0.01).to(DT[io]), rnd(m, n, std=2.0).to(DT[io]), rnd(m, n).to(DT[io])
    for i, act in enumerate(ACTS):
        bias = i % 2 == 0
        for path, got in paths_for(lambda p: native.w4a8_glu_grad(dh, g, u, wg, sg, wu, su, k, act=act,
                                                                  bias_grad=bias, path=p)):
            want, db = ref.glu_grad(dh, g, u, qg, sg, qu, su, act, path == "tc")
            for t, w, what in zip(got if bias else (got,), [want] + db, ("dx", "dbg", "dbu")):
                ref.check(t, *w, f"{what} {act} {path}")


def test_float32_gradient_keeps_its_second_term():
    """With few terms in the sum the bound of a float32 gradient is far below
    one FP16 rounding of the rows (2^-11)."""
    rnd = gen(3)
    q, sw, wp = weights(rnd, 8, 200)
    dy = rnd(150, 8)
    for path, got in paths_for(lambda p: native.w4a8_linear_act_grad(dy, wp, sw, 200, path=p)):
        (dx, e), _ = ref.linear_grad(dy, dy, q, sw, "none", path == "tc")
        assert float((e / (dy.double().abs() / sw.double()).matmul(q.double().abs()).clamp(min=1e-30)).max()) < 2.0 ** -16
        ref.check(got, dx, e, path)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(3, 200, 90), (40, 200, 90), (200, 328, 200)])
def test_row_strides_and_neighbours(io, m, k, n):
    """Rows inside wider buffers, at offsets that are not 16-byte aligned, give
    the same results, and nothing beside the rows is written."""
    rnd, dt = gen(m + n), DT[io]
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    # weight rows of a wider stride
    wide = torch.full((2, n, wg.shape[1] + 32), 0x77, dtype=torch.uint8, device="cuda")
    wide[0, :, : wg.shape[1]], wide[1, :, : wu.shape[1]] = wg, wu
    wgs, wus = wide[0], wide[1]

    def inside(t, off, pad):
        buf = torch.full((t.shape[0] + 2, t.shape[1] + pad + off), 7.0, dtype=dt, device="cuda")
        v = buf[1:-1, off: off + t.shape[1]]
        v.copy_(t)
        return buf, v

    def untouched(buf, v):
        v.fill_(7.0)
        assert (buf == 7.0).all()

    x, dh = rows(rnd, m, k, dt), rnd(m, n).to(dt)
    want_h = ref.glu(x, qg, sg, qu, su, None, None, "silu")
    want_y = ref.linear(x, qg, sg, None, "gelu_tanh", dh)
    for off, pad in ((0, 8), (1, 0), (3, 5), (8, 24)):
        _, xv = inside(x, off, pad)
        outs = [inside(torch.zeros(m, n, device="cuda"), off, pad) for _ in range(3)]
        got = native.w4a8_glu(xv, wgs, sg, wus, su, h=outs[0][1], g=outs[1][1], u=outs[2][1])
        for t, (w, e), what in zip(got, want_h, "hgu"):
            ref.check(t, w, e, f"{what} off {off}")
        g, u = inside(got[1], off, pad)[1], inside(got[2], off, pad)[1]
        for o in outs:
            untouched(*o)
        by, yv = inside(dh, off, pad)                      # the residual in place
        ref.check(native.w4a8_linear_act(xv, wgs, sg, act="gelu_tanh", residual=yv, y=yv), *want_y[0], "y in place")
        untouched(by, yv)
        bd, dxv = inside(torch.zeros(m, k, device="cuda"), off, pad)
        _, dhv = inside(dh, off, pad)
        got = native.w4a8_glu_grad(dhv, g, u, wgs, sg, wus, su, k, dx=dxv)
        want, _ = ref.glu_grad(dhv, g, u, qg, sg, qu, su, "silu", native.last_path() == "tc")
        ref.check(got, *want, f"dx off {off}")
        untouched(bd, dxv)


def test_zero_rows_and_columns():
    """A zero row gives z = bias, a zero weight channel too; a zero gradient
    row gives zeros."""
    rnd = gen(9)
    for m in (1, 6, 150):
        q, sw, wp = weights(rnd, 70, 100)
        q[3] = 0
        sw[3] = 1.0
        wp = ref.pack(q)
        x, b = rnd(m, 100), rnd(70)
        x[0] = 0.0
        y, z = native.w4a8_linear_act(x, wp, sw, bias=b, act="silu", save=True)
        assert torch.equal(z[0], b) and torch.equal(z[:, 3], b[3].expand(m))
        dy = rnd(m, 70)
        dy[-1] = 0.0
        dx = native.w4a8_linear_act_grad(dy, wp, sw, 100, act="silu", z=z)
        assert (dx[-1] == 0).all() and torch.isfinite(dx).all()


def test_saturated_activations():
    """Pre-activations far into both tails stay finite and exact to the bounds."""
    rnd = gen(10)
    n, k, m = 64, 40, 33
    q, sw, wp = weights(rnd, n, k)
    x = rnd(m, k)
    b = torch.linspace(-300.0, 300.0, n, device="cuda")
    z = (b + torch.zeros(m, 1, device="cuda")).contiguous()
    dy = rnd(m, n)
    for act in ACTS:
        got = native.w4a8_linear_act(x, wp, sw, bias=b, act=act)
        ref.check(got, *ref.linear(x, q, sw, b, act, None)[0], act)
        (dx, e), _ = ref.linear_grad(dy, z, q, sw, act, False)
        ref.check(native.w4a8_linear_act_grad(dy, wp, sw, k, act=act, z=z), dx, e, act)
        u = rnd(m, n)
        (dx, e), _ = ref.glu_grad(dy, z, u, q, sw, q, sw, act, False)
        ref.check(native.w4a8_glu_grad(dy, z, u, wp, sw, wp, sw, k, act=act), dx, e, act)


def test_gradient_rows_of_very_different_size():
    """Each row has its own power of two: tiny and huge rows keep their precision."""
    rnd = gen(12)
    q, sw, wp = weights(rnd, 96, 80)
    dy = rnd(64, 96) * (2.0 ** torch.linspace(-100, 80, 64, device="cuda"))[:, None]
    for path, got in paths_for(lambda p: native.w4a8_linear_act_grad(dy, wp, sw, 80, path=p)):
        want, _ = ref.linear_grad(dy, dy, q, sw, "none", path == "tc")
        ref.check(got, *want, path)


def test_no_rows():
    wp, sw = torch.zeros((5, 16), dtype=torch.uint8, device="cuda"), torch.ones(5, device="cuda")
    x = torch.zeros((0, 9), device="cuda")
    assert native.w4a8_linear_act(x, wp, sw).shape == (0, 5)
    h, g, u = native.w4a8_glu(x, wp, sw, wp, sw, save=True)
    assert h.shape == g.shape == u.shape == (0, 5)
    dx, a, b = native.w4a8_glu_grad(h, g, u, wp, sw, wp, sw, 9, bias_grad=True)
    assert dx.shape == (0, 9) and (a == 0).all() and (b == 0).all()
    dx, a = native.w4a8_linear_act_grad(h, wp, sw, 9, bias_grad=True)
    assert dx.shape == (0, 9) and (a == 0).all()


def block(x, p, act, kw=()):
    """A gated feed-forward block with its residual, forward and backward."""
    kw = dict(kw)
    h, g, u = native.w4a8_glu(x, *p["g"], *p["u"], act=act, save=True, **kw)
    y = native.w4a8_linear_act(h, *p["d"], residual=x, **kw)
    dh = native.w4a8_linear_act_grad(y, *p["d"], h.shape[1], **kw)
    dx = native.w4a8_glu_grad(dh, g, u, *p["g"], *p["u"], x.shape[1], act=act, **kw)
    return h, g, u, y, dh, dx


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 7, 16, 33, 700])
def test_whole_block(io, m):
    """The operators as a block runs them, each stage checked on the stage
    before it, with a second run on another stream giving the same bits."""
    d, f, act = 192, 520, "gelu_tanh"
    rnd = gen(m)
    q, p = {}, {}
    for name, (n, k) in dict(g=(f, d), u=(f, d), d=(d, f)).items():
        qq, sw, wp = weights(rnd, n, k)
        q[name], p[name] = (qq, sw), (wp, sw)
    x = rows(rnd, m, d, DT[io])
    h, g, u, y, dh, dx = first = block(x, p, act, dict(static_weights=True))
    for t, (w, e), what in zip((h, g, u), ref.glu(x, *q["g"], *q["u"], None, None, act), "hgu"):
        ref.check(t, w, e, what)
    ref.check(y, *ref.linear(h, *q["d"], None, "none", x)[0], "y")
    ref.check(dh, *ref.linear_grad(y, y, *q["d"], "none", False)[0], "dh")
    ref.check(dx, *ref.glu_grad(dh, g, u, *q["g"], *q["u"], act, False)[0], "dx")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = block(x, p, act)
    s.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_captured_blocks_replay():
    """Two graphs of the block, captured with their own workspaces and replayed
    in turn with new inputs in place, give the eager results."""
    d, f = 96, 260
    rnd = gen(2)
    p = {}
    for name, (n, k) in dict(g=(f, d), u=(f, d), d=(d, f)).items():
        _, sw, wp = weights(rnd, n, k)
        p[name] = (wp, sw)
    xs = [rows(rnd, m, d, torch.bfloat16) for m in (2, 150)]
    block(xs[0], p, "silu"), block(xs[1], p, "silu")       # first calls outside the capture
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(block(x, p, "silu"))
        graphs.append(g)
    for seed in range(3):
        r = gen(100 + seed)
        for x in xs:
            x.copy_(rows(r, x.shape[0], d, torch.bfloat16))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, out in zip(xs, outs):
            for a, b in zip(out, block(x, p, "silu")):
                assert torch.equal(a, b)


def test_bias_gradients_repeat_and_cover_many_rows():
    rnd = gen(6)
    q, sw, wp = weights(rnd, 100, 64)
    dy = rnd(1500, 100).bfloat16()
    runs = [native.w4a8_linear_act_grad(dy, wp, sw, 64, bias_grad=True) for _ in range(2)]
    (dx, e), db = ref.linear_grad(dy, dy, q, sw, "none", False)
    ref.check(runs[0][0], dx, e, "dx")
    ref.check(runs[0][1], *db[0], "db")
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_offsets_past_32_bits():
    """Rows so far apart that their byte offsets pass 2^32."""
    ld, m, k, n = 1 << 30, 3, 72, 40
    rnd = gen(8)
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    buf = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda")
    at = lambda cols, off: buf.as_strided((m, cols), (ld, 1), off)
    x, h, g, u, dx = at(k, 0), at(n, 1000), at(n, 2000), at(n, 3000), at(k, 4000)
    x.copy_(rows(rnd, m, k, torch.bfloat16))
    native.w4a8_glu(x, wg, sg, wu, su, h=h, g=g, u=u)
    for t, (w, e), what in zip((h, g, u), ref.glu(x, qg, sg, qu, su, None, None, "silu"), "hgu"):
        ref.check(t, w, e, what)
    native.w4a8_glu_grad(h, g, u, wg, sg, wu, su, k, dx=dx)
    ref.check(dx, *ref.glu_grad(h, g, u, qg, sg, qu, su, "silu", False)[0], "dx")


def test_huge_finite_preactivations():
    """Finite pre-activations of any size give finite values: the activations'
    limits and derivatives 0 or 1."""
    n, k = 16, 8
    q = torch.zeros((n, k), dtype=torch.int8, device="cuda")
    q[:, 0] = 7
    wp, sw = ref.pack(q), torch.ones(n, device="cuda")
    b = torch.tensor([1e30, -1e30, 1e20, -1e20, 3e4, -3e4, 200.0, -200.0] * 2, device="cuda")
    x = torch.zeros((3, k), device="cuda")
    for act in ACTS[1:]:
        y, z = native.w4a8_linear_act(x, wp, sw, bias=b, act=act, save=True)
        assert torch.equal(z, b.expand(3, n))
        assert torch.equal(y, torch.where(b > 0, b, torch.zeros_like(b)).expand(3, n)), act
        dx = native.w4a8_linear_act_grad(torch.ones(3, n, device="cuda"), wp, sw, k, act=act, z=z)
        assert torch.equal(dx[:, 0], torch.full((3,), 7.0 * 8, device="cuda")) and (dx[:, 1:] == 0).all(), act


@pytest.mark.parametrize("m,k,n,io", [(100, 1152, 333, "f32"), (500, 1152, 1000, "f32"), (500, 1152, 1000, "bf16"),
                                      (40, 4096, 2000, "bf16"), (12, 1152, 6912, "bf16"), (1, 4096, 4096, "f32")])
def test_many_calls_give_the_same_bits(m, k, n, io):
    """Two hundred calls in a row, as overlapped as the stream allows, repeat
    the first one's bits: every hand-over between the kernels' warps holds."""
    rnd = gen(m + n)
    (_, sg, wg), (_, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    x, dh = rows(rnd, m, k, DT[io]), rnd(m, n, std=0.01).to(DT[io])
    h, g, u = native.w4a8_glu(x, wg, sg, wu, su, save=True)
    for call in (lambda: native.w4a8_glu(x, wg, sg, wu, su, static_weights=True),
                 lambda: native.w4a8_linear_act(x, wg, sg, act="silu", residual=dh),
                 lambda: native.w4a8_glu_grad(dh, g, u, wg, sg, wu, su, k),
                 lambda: native.w4a8_linear_act_grad(dh, wg, sg, k, act="silu", z=g)):
        first = call()
        again = [call() for _ in range(200)]
        assert all(torch.equal(first, a) for a in again)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradients_of_very_wide_layers(io):
    """Rows whose values exceed a block's shared memory."""
    rnd, m, k = gen(21), 3, 40
    for n, glu in ((56400, False), (28300, True)):
        (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
        dh, g, u = rnd(m, n, std=0.01).to(DT[io]), rnd(m, n).to(DT[io]), rnd(m, n).to(DT[io])
        if glu:
            got = native.w4a8_glu_grad(dh, g, u, wg, sg, wu, su, k)
            want, _ = ref.glu_grad(dh, g, u, qg, sg, qu, su, "silu", True)
        else:
            got = native.w4a8_linear_act_grad(dh, wg, sg, k, act="silu", z=g)
            want, _ = ref.linear_grad(dh, g, qg, sg, "silu", True)
        ref.check(got, *want, f"N = {n}")


def test_longest_sums():
    """K at its limit (the largest INT32 sums) and rows longer than a block
    holds, few rows and many."""
    rnd, k, n = gen(22), native.ACT_MAX_K, 24
    q, sw, wp = weights(rnd, n, k)
    q[:2] = 7                       # codes and rows at their largest: |16 acc| just below 2^31
    wp, x = ref.pack(q), None
    for m in (1, 40):
        x = rnd(m, k)
        x[0] = 1.0
        want = ref.linear(x, q, sw, None, "none", None)[0]
        for path, got in paths_for(lambda p: native.w4a8_linear_act(x, wp, sw, path=p)):
            ref.check(got, *want, f"m {m} {path}")
    with pytest.raises(native.W4A8Error):
        native.w4a8_linear_act(torch.zeros(1, k + 1, device="cuda"),
                               torch.zeros(1, native.packed_ld(k + 1), dtype=torch.uint8, device="cuda"),
                               torch.ones(1, device="cuda"))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [520, 523])
def test_shared_tiles(io, n):
    """Long sums over few tiles: the pairs share the stages out and a third
    launch joins the parts and finishes, whatever the epilogue."""
    m, k = 40, 16390
    rnd = gen(n)
    (qg, sg, wg), (qu, su, wu) = weights(rnd, n, k), weights(rnd, n, k)
    x, r, b1, b2 = rows(rnd, m, k, DT[io]), rnd(m, n, std=2.0).to(DT[io]), rnd(n), rnd(n)
    for act in ACTS:
        got = native.w4a8_linear_act(x, wg, sg, bias=b1, act=act, residual=r, save=True, path="tc")
        assert native.last_launch_count() == 3
        for t, (w, e), what in zip(got, ref.linear(x, qg, sg, b1, act, r), "yz"):
            ref.check(t, w, e, f"{what} {act}")
        got = native.w4a8_glu(x, wg, sg, wu, su, gate_bias=b1, up_bias=b2, act=act, save=True, path="tc")
        assert native.last_launch_count() == 3
        for t, (w, e), what in zip(got, ref.glu(x, qg, sg, qu, su, b1, b2, act), "hgu"):
            ref.check(t, w, e, f"{what} {act}")
    dh = rnd(m, k, std=0.01).to(DT[io])       # the same layer the other way round: N and K exchanged
    q, sw, wp = weights(rnd, k, n)
    got = native.w4a8_linear_act_grad(dh, wp, sw, n)
    assert native.last_launch_count() == 3
    ref.check(got, *ref.linear_grad(dh, dh, q, sw, "none", True)[0], "dx")


def test_two_streams_at_once():
    """Blocks running on two streams at the same time, each with its own
    buffers, give the bits they give alone."""
    d, f = 512, 1300
    rnd = gen(31)
    p = {}
    for name, (n, k) in dict(g=(f, d), u=(f, d), d=(d, f)).items():
        _, sw, wp = weights(rnd, n, k)
        p[name] = (wp, sw)
    xs = [rows(rnd, m, d, dt) for m, dt in ((300, torch.bfloat16), (5, torch.float32))]
    alone = [block(x, p, "silu") for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    both = []
    for _ in range(20):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                both.append(block(x, p, "silu"))
    torch.cuda.synchronize()
    for i, out in enumerate(both):
        for a, b in zip(alone[i % 2], out):
            assert torch.equal(a, b)

"""The dense linear with its epilogue (dense_forward, dense_backward,
DenseLinear) against plain float64 formulas, element by element.

Tolerances, per element, with half = eps / 2 of the output type (bf16 2^-8,
float32 2^-24) and s = the product of absolute values that the sum runs over:
  a float32 sum of n products     2 (n + 8) 2^-24 s   (order unknown; twice the
                                  bound of recursive summation, for partial
                                  sums inside the matrix instruction)
  an output rounding              half |value|
  g_u as a bf16 operand           half s once more
  activation                      slopes are at most 1.13 in size, and the
                                  formula's own float32 steps err by at most
                                  1e-6 max(1, |u|)
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here is gpu-marked
    pytest.skip("no GPU", allow_module_level=True)

from orthogonal_equivalence_amd import poetx as P  # noqa: E402
from orthogonal_equivalence_amd.dense import (ACTIVATIONS, DenseLinear,  # noqa: E402
                                              dense_backward, dense_forward)

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
ACTS = tuple(ACTIVATIONS)


def act64(u, name):
    """act(u) and its slope in float64."""
    if name == "relu":
        return u.clamp(min=0), (u > 0).double()
    if name == "gelu":
        cdf = torch.special.ndtr(u)
        return u * cdf, cdf + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c, a = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(c * (u + a * u ** 3))
        return 0.5 * u * (1 + t), 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * c * (1 + 3 * a * u * u)
    if name == "silu":
        p = torch.sigmoid(u)
        return u * p, p * (1 + u * (1 - p))
    return u, torch.ones_like(u)


def make(tokens, d_in, d_out, dtype, seed=0, int8=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, k=1.0: torch.randn(*s, generator=g, device="cuda") * k  # noqa: E731
    dt = DT[dtype]
    t = dict(x=rnd(tokens, d_in).to(dt), W=rnd(d_out, d_in, k=d_in ** -0.5).to(dt), w_scale=None,
             bias=rnd(d_out, k=0.5), residual=rnd(tokens, d_out).to(dt),
             g_y=rnd(tokens, d_out, k=0.1).to(dt), u=rnd(tokens, d_out, k=1.5).to(dt))
    if int8:
        t["W"] = torch.randint(-127, 128, (d_out, d_in), generator=g, device="cuda",
                               dtype=torch.int8)
        t["w_scale"] = (0.5 + torch.rand(d_out, generator=g, device="cuda")) / (73 * d_in ** 0.5)
    return t


def weight64(t):
    W = t["W"].double()
    return W if t["w_scale"] is None else W * t["w_scale"].double()[:, None]


def close(name, got, ref, tol):
    assert got.shape == ref.shape, name
    err = (got.double() - ref).abs()
    worst = (err / tol.clamp(min=1e-300)).max().item()
    print(f"    {name}: worst error / tolerance {worst:.3f}", flush=True)
    assert torch.isfinite(got).all(), name
    assert worst <= 1.0, (name, worst)


def check_forward(t, dtype, act, bias=True, residual=True):
    half = HALF[dtype]
    b = t["bias"] if bias else None
    r = t["residual"] if residual else None
    y, u = dense_forward(t["x"], t["W"], b, r, act, t["w_scale"], save_u=True)
    y2, none = dense_forward(t["x"], t["W"], b, r, act, t["w_scale"])
    assert none is None and torch.equal(y, y2)  # the same with and without u, and twice
    x, W = t["x"].double(), weight64(t)
    u64 = x @ W.t()
    s = x.abs() @ W.abs().t()
    if bias:
        u64, s = u64 + b.double(), s + b.double().abs()
    y64 = act64(u64, act)[0]
    err = 2 * (x.shape[1] + 8) * 2.0 ** -24 * s
    close("u", u, u64, err + half * (u64.abs() + err))
    err = 1.13 * err + (1e-6 * u64.abs().clamp(min=1) if act != "none" else 0)
    if residual:
        y64 = y64 + r.double()
        err = err + 2.0 ** -23 * (y64.abs() + r.double().abs())
    close("y", y, y64, err + half * (y64.abs() + err))


def check_backward(t, dtype, act, g_W=True):
    half = HALF[dtype]
    n = t["g_y"].shape
    gx, gW, gb = dense_backward(t["g_y"], t["W"], t["x"], t["u"], act, t["w_scale"],
                                need_g_W=g_W, need_g_bias=True)
    g = t["g_y"].double()
    slope = act64(t["u"].double(), act)[1]
    gu = g * slope
    # g_u's own error: the slope's formula, one product
    eu = (1e-6 * t["u"].double().abs().clamp(min=1) * g.abs() if act != "none" else 0 * g)
    eb = eu.sum(0) + (n[0] + 8) * 2.0 ** -23 * gu.abs().sum(0)
    close("g_bias", gb, gu.sum(0), eb + 2.0 ** -24 * gu.sum(0).abs() + 1e-30)
    # the operand's rounding (none where g_y itself is the operand)
    op = half if act != "none" or t["w_scale"] is not None else 0.0
    W = weight64(t)
    s = gu.abs() @ W.abs()
    e = (eu + 2 * op * gu.abs()) @ W.abs() + 2 * (n[1] + 8) * 2.0 ** -24 * s
    ref = gu @ W
    close("g_x", gx, ref, e + half * (ref.abs() + e) + 1e-30)
    if g_W:
        x = t["x"].double()
        s = gu.abs().t() @ x.abs()
        e = (eu + 2 * op * gu.abs()).t() @ x.abs() + 2 * (n[0] + 8) * 2.0 ** -24 * s
        ref = gu.t() @ x
        close("g_W", gW, ref, e + half * (ref.abs() + e) + 1e-30)
    else:
        assert gW is None


# tokens, d_in, d_out: one token to several tiles; widths at, below and past
# the tiles and the reduction steps (64 bf16, 32 float32), long reductions
# that are split, single vectors
SIZES = [(1, 8, 8), (1, 128, 128), (1, 4096, 256), (2, 136, 264), (3, 2056, 72), (7, 512, 1024),
         (16, 1000, 520), (17, 64, 4096), (31, 4096, 512), (33, 8192, 128), (63, 256, 256),
         (64, 72, 8), (65, 320, 192), (100, 1024, 1536), (127, 256, 640), (128, 512, 128),
         (129, 2048, 256), (200, 1000, 136), (255, 512, 520), (256, 256, 256), (257, 512, 768),
         (300, 2056, 1288), (513, 1024, 2048), (777, 2048, 1024), (1100, 768, 2816),
         # INT8 rows of whole 16 bytes that end inside a step; a long split
         (5, 144, 136), (20, 14336, 96), (40, 144, 136), (90, 1040, 264), (150, 4112, 512)]


@pytest.mark.parametrize("i", range(len(SIZES)), ids=lambda i: "x".join(map(str, SIZES[i])))
@pytest.mark.parametrize("dtype", ["bf16", "f32", "int8"])
def test_forward(i, dtype):
    tokens, d_in, d_out = SIZES[i]
    int8 = dtype == "int8"
    dt = "bf16" if int8 else dtype
    t = make(tokens, d_in, d_out, dt, seed=i, int8=int8)
    for k in range(2):
        act, bias, res = ACTS[(i + 2 * k) % 5], (i + k) % 2 == 0, (i // 2 + k) % 2 == 0
        print(f"  {tokens}x{d_in}x{d_out} {dtype} {act} bias={bias} residual={res}", flush=True)
        check_forward(t, dt, act, bias, res)


@pytest.mark.parametrize("i", range(len(SIZES)), ids=lambda i: "x".join(map(str, SIZES[i])))
@pytest.mark.parametrize("dtype", ["bf16", "f32", "int8"])
def test_backward(i, dtype):
    tokens, d_in, d_out = SIZES[i]
    int8 = dtype == "int8"
    dt = "bf16" if int8 else dtype
    t = make(tokens, d_in, d_out, dt, seed=100 + i, int8=int8)
    for k in range(2):
        act = ACTS[(i + 2 * k) % 5]
        print(f"  {tokens}x{d_in}x{d_out} {dtype} {act}", flush=True)
        check_backward(t, dt, act, g_W=not int8)


# products large enough for the 256 x 256 tiles, whole (the tiled layouts of
# INT8 codes and of g_u) and ragged in rows, columns and both reductions
@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("tokens,d_in,d_out", [(4096, 1024, 4096), (4096, 4096, 1024),
                                               (4200, 1056, 4360), (4333, 4360, 1056),
                                               (2048, 4096, 14336)])
def test_large(tokens, d_in, d_out, dtype):
    int8 = dtype == "int8"
    t = make(tokens, d_in, d_out, "bf16", seed=41, int8=int8)
    print(f"  {tokens}x{d_in}x{d_out} {dtype}", flush=True)
    check_forward(t, "bf16", "silu")
    check_forward(t, "bf16", "none", bias=False)
    check_backward(t, "bf16", "gelu", g_W=False)
    check_backward(t, "bf16", "none", g_W=not int8)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_activation(act, dtype):
    t = make(70, 256, 384, dtype, seed=7)
    check_forward(t, dtype, act)
    check_backward(t, dtype, act)


def test_int8_with_float32_activations():
    t = make(37, 264, 136, "f32", seed=8, int8=True)
    check_forward(t, "f32", "silu")
    check_backward(t, "f32", "silu", g_W=False)


@pytest.mark.parametrize("act", ACTS)
def test_activation_at_far_arguments(act):
    """u = bias (x = 0): large, tiny and zero arguments; the slopes too."""
    v = [0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 0.5, -0.5, 3.0, -3.0, 9.0, -9.0, 20.0, -20.0,
         90.0, -90.0, 1e4, -1e4, 1e18, -1e18, 3e38, -3e38, 12.5, -12.5]
    bias = torch.tensor(v, device="cuda")
    x = torch.zeros(3, 8, device="cuda")
    W = torch.zeros(len(v), 8, device="cuda")
    y, u = dense_forward(x, W, bias, activation=act, save_u=True)
    assert torch.equal(u, bias.expand(3, -1))
    y64, slope = act64(bias.double().clamp(-1e18, 1e18), act)
    y64 = torch.where(bias.double().abs() > 1e18, act64(bias.double().sign(), "relu")[0]
                      * bias.double() if act != "none" else bias.double(), y64)
    tol = 1e-6 * bias.double().abs().clamp(min=1) + 2.0 ** -24 * y64.abs()
    assert torch.isfinite(y).all()
    assert ((y.double() - y64).abs() <= tol).all(), (y[0], y64)
    g = torch.ones(3, len(v), device="cuda")
    _, _, gb = dense_backward(g, W, u=u, activation=act, need_g_x=False, need_g_bias=True)
    slope = torch.where(bias.abs() > 80, (bias > 0).double() if act != "none" else slope, slope)
    assert ((gb.double() - 3 * slope).abs() <= 3e-5).all(), (gb, 3 * slope)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 5, 70, 300])
def test_nan_and_infinity_stay_in_their_row_and_column(dtype, tokens):
    t = make(tokens, 264, 328, dtype, seed=11)
    ref, _ = dense_forward(t["x"], t["W"], t["bias"], activation="gelu")
    x, W, bias = t["x"].clone(), t["W"].clone(), t["bias"].clone()
    x[tokens - 1, 263] = float("nan")
    W[327, 263] = float("nan")
    bias[5] = float("inf")
    y, _ = dense_forward(x, W, bias, activation="gelu")
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[tokens - 1] = True
    hit[:, 327] = True
    assert torch.isnan(y[hit]).all()
    keep = ~hit
    keep[:, 5] = False
    assert torch.equal(y[keep], ref[keep])
    assert torch.isinf(y[:tokens - 1, 5]).all()
    # the backward: a NaN gradient row reaches g_x's row, g_W and g_bias columns
    g_y = t["g_y"].clone()
    g_y[tokens - 1, 3] = float("nan")
    gx, gW, gb = dense_backward(g_y, t["W"], t["x"], t["u"], "silu", need_g_W=True,
                                need_g_bias=True)
    rx, rW, rb = dense_backward(t["g_y"], t["W"], t["x"], t["u"], "silu", need_g_W=True,
                                need_g_bias=True)
    assert torch.isnan(gx[tokens - 1]).all() and torch.equal(gx[:tokens - 1], rx[:tokens - 1])
    rows = torch.arange(328, device="cuda") != 3
    assert torch.isnan(gW[3]).all() and torch.equal(gW[rows], rW[rows])
    assert torch.isnan(gb[3]) and torch.equal(gb[rows], rb[rows])


@pytest.mark.parametrize("tokens,d_in,d_out", [(1, 256, 136), (65, 200, 264), (300, 1288, 520)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_is_written_outside_the_outputs(tokens, d_in, d_out, dtype):
    """Outputs inside larger buffers of a sentinel, workspace of the exact size
    between guards."""
    t = make(tokens, d_in, d_out, dtype, seed=13)
    pad = 1024

    def guarded(n, dt, value):
        buf = torch.full((n + 2 * pad,), value, device="cuda", dtype=dt)
        return buf, buf[pad:pad + n]

    def whole(buf, n, value):
        return bool((buf[:pad] == value).all()) and bool((buf[pad + n:] == value).all())

    act = P.POETX_BF16 if dtype == "bf16" else P.POETX_F32
    desc = P.make_dense_desc(tokens, d_in, d_out, act, P.POETX_ACT_SILU)
    fw, bw = P.poetx_dense_fwd_workspace_size(desc), P.poetx_dense_bwd_workspace_size(desc)
    wbuf, ws = guarded(max(fw, bw), torch.uint8, 77)
    dt = DT[dtype]
    ybuf, y = guarded(tokens * d_out, dt, 7.0)
    ubuf, u = guarded(tokens * d_out, dt, 7.0)
    P.poetx_dense_fwd(desc, t["x"], t["W"], t["bias"], t["residual"], y, u,
                      ws[:fw] if fw else None)
    xbuf, gx = guarded(tokens * d_in, dt, 7.0)
    gbuf, gW = guarded(d_out * d_in, dt, 7.0)
    bbuf, gb = guarded(d_out, torch.float32, 7.0)
    P.poetx_dense_bwd(desc, t["g_y"], t["x"], t["W"], u, gx, gW, gb, ws[:bw])
    torch.cuda.synchronize()
    for buf, n, v in ((ybuf, tokens * d_out, 7.0), (ubuf, tokens * d_out, 7.0),
                      (xbuf, tokens * d_in, 7.0), (gbuf, d_out * d_in, 7.0), (bbuf, d_out, 7.0),
                      (wbuf, max(fw, bw), 77)):
        assert whole(buf, n, v)
    ry, ru = dense_forward(t["x"], t["W"], t["bias"], t["residual"], "silu", save_u=True)
    assert torch.equal(y.view(tokens, d_out), ry) and torch.equal(u.view(tokens, d_out), ru)
    rx, rW, rb = dense_backward(t["g_y"], t["W"], t["x"], ru, "silu", need_g_W=True,
                                need_g_bias=True)
    assert torch.equal(gx.view(tokens, d_in), rx) and torch.equal(gW.view(d_out, d_in), rW)
    assert torch.equal(gb, rb)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """float32 gradients along one direction against the central difference
    of the float64 loss sum(g_y y): step h = 1e-5 in float64 leaves an h^2
    term below 1e-8; the gradients' float32 sums are good to 1e-5."""
    t = make(33, 72, 104, "f32", seed=17)
    x, W, b, r, g = (t[k].double() for k in ("x", "W", "bias", "residual", "g_y"))
    gen = torch.Generator(device="cuda").manual_seed(3)
    dx, dW, db = (torch.randn(v.shape, generator=gen, device="cuda").double() for v in (x, W, b))

    def loss(h):
        u = (x + h * dx) @ (W + h * dW).t() + b + h * db
        if act == "relu":  # the side of zero of the middle point (no kink inside the step)
            return (torch.where(x @ W.t() + b > 0, u, 0 * u) * g).sum()
        return (act64(u, act)[0] * g).sum()

    h = 1e-5
    diff = ((loss(h) - loss(-h)) / (2 * h)).item()
    _, u = dense_forward(t["x"], t["W"], t["bias"], t["residual"], act, save_u=True)
    gx, gW, gb = dense_backward(t["g_y"], t["W"], t["x"], u, act, need_g_W=True, need_g_bias=True)
    terms = [(gx.double() * dx).sum(), (gW.double() * dW).sum(), (gb.double() * db).sum()]
    size = sum((a.double().abs() * b.abs()).sum().item() for a, b in ((gx, dx), (gW, dW), (gb, db)))
    got = sum(v.item() for v in terms)
    print(f"    {act}: difference {diff:.6f}, gradients {got:.6f}", flush=True)
    assert abs(got - diff) <= 1e-5 * size + 1e-6


def test_outputs_that_are_not_asked_for():
    t = make(40, 128, 136, "bf16", seed=19)
    full = dense_backward(t["g_y"], t["W"], t["x"], t["u"], "silu", need_g_W=True, need_g_bias=True)
    only = [dense_backward(t["g_y"], t["W"], u=t["u"], activation="silu"),
            dense_backward(t["g_y"], t["W"], t["x"], t["u"], "silu", need_g_x=False, need_g_W=True),
            dense_backward(t["g_y"], t["W"], u=t["u"], activation="silu", need_g_x=False,
                           need_g_bias=True)]
    for k, o in enumerate(only):
        for j in range(3):
            assert (o[j] is None) == (j != k)
        assert torch.equal(o[k], full[k])


def test_other_stream_and_graph():
    """The call on a side stream, and captured into a graph that is replayed
    several times on new inputs between eager calls."""
    t = make(150, 256, 392, "bf16", seed=23)
    ref = dense_forward(t["x"], t["W"], t["bias"], t["residual"], "silu", save_u=True)
    refb = dense_backward(t["g_y"], t["W"], t["x"], ref[1], "silu", need_g_W=True, need_g_bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = dense_forward(t["x"], t["W"], t["bias"], t["residual"], "silu", save_u=True, stream=s)
    sideb = dense_backward(t["g_y"], t["W"], t["x"], side[1], "silu", need_g_W=True,
                           need_g_bias=True, stream=s)
    handle = dense_forward(t["x"], t["W"], t["bias"], t["residual"], "silu", stream=s.cuda_stream)
    null = dense_forward(t["x"], t["W"], t["bias"], t["residual"], "silu", stream=0)
    torch.cuda.synchronize()
    assert torch.equal(null[0], ref[0])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*ref, *refb, ref[0]), (*side, *sideb, handle[0])))

    x, g_y = t["x"].clone(), t["g_y"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, u = dense_forward(x, t["W"], t["bias"], t["residual"], "silu", save_u=True)
        grads = dense_backward(g_y, t["W"], x, u, "silu", need_g_W=True, need_g_bias=True)
    for k in range(4):
        n = make(150, 256, 392, "bf16", seed=50 + k)
        x.copy_(n["x"])
        g_y.copy_(n["g_y"])
        graph.replay()
        ey, eu = dense_forward(n["x"], t["W"], t["bias"], t["residual"], "silu", save_u=True)
        eg = dense_backward(n["g_y"], t["W"], n["x"], eu, "silu", need_g_W=True, need_g_bias=True)
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(u, eu)
        assert all(torch.equal(a, b) for a, b in zip(grads, eg))


def test_dense_linear():
    t = make(50, 264, 200, "bf16", seed=29)
    lay = DenseLinear(t["W"].float().cpu(), "bf16", t["bias"].cpu(), "gelu")
    y, u = lay.forward(t["x"], t["residual"], save_u=True)
    ry, ru = dense_forward(t["x"], t["W"], t["bias"], t["residual"], "gelu", save_u=True)
    assert torch.equal(y, ry) and torch.equal(u, ru)
    gx, gW, gb = lay.backward(t["g_y"], t["x"], u, need_g_W=True)
    rx, rW, rb = dense_backward(t["g_y"], t["W"], t["x"], ru, "gelu", need_g_W=True,
                                need_g_bias=True)
    assert torch.equal(gx, rx) and torch.equal(gW, rW) and torch.equal(gb, rb)
    # INT8: within the codes' half step (scale / 2 an element) of the bf16 layer
    q = DenseLinear(t["W"], "bf16", int8=True)
    yq, _ = q.forward(t["x"])
    y0 = t["x"].double() @ t["W"].double().t()
    tol = 0.501 * q.w_scale.double() * t["x"].double().abs().sum(1, keepdim=True)
    assert ((yq.double() - y0).abs() <= tol + 2.0 ** -7 * y0.abs()).all()


def test_refusals():
    t = make(10, 64, 72, "bf16")
    for bad in (dict(bias=t["bias"].bfloat16()), dict(bias=t["bias"][:64]),
                dict(residual=t["x"]), dict(residual=t["residual"].float()),
                dict(activation="tanh"), dict(w_scale=torch.ones(72, device="cuda")),
                dict(residual=t["residual"].cpu())):
        with pytest.raises(ValueError):
            dense_forward(t["x"], t["W"], **bad)
    for x, W in ((t["x"].t(), t["W"]), (t["x"].half(), t["W"].half()), (t["x"], t["W"].t()),
                 (t["x"][0], t["W"]), (t["x"].cpu(), t["W"].cpu())):
        with pytest.raises(ValueError):
            dense_forward(x, W)
    with pytest.raises(ValueError):  # a view with other strides
        dense_forward(torch.zeros(10, 128, device="cuda", dtype=torch.bfloat16)[:, ::2], t["W"])
    with pytest.raises(P.PoetxError):  # no rows
        dense_forward(t["x"][:0], t["W"])
    with pytest.raises(P.PoetxError):  # width not a multiple of 8
        dense_forward(t["x"][:, :60].contiguous(), t["W"][:, :60].contiguous())
    for bad in (dict(need_g_W=True), dict(activation="silu"), dict(need_g_x=False),
                dict(x=t["x"], w_scale=torch.ones(72, device="cuda"), need_g_W=True)):
        with pytest.raises(ValueError):
            dense_backward(t["g_y"], t["W"], **bad)

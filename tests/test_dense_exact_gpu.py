"""The dense linear on operands of small integers, bit for bit: every product
and sum is exact in float32 in any order, so an output is the exact value
rounded once to its type, on every kernel variant that the plans choose
(dense_cases.py) and past 2^32 elements, where every element is compared."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here is gpu-marked
    pytest.skip("no GPU", allow_module_level=True)

from orthogonal_equivalence_amd.dense import dense_backward, dense_forward  # noqa: E402
from tests.dense_cases import BF16, CASES, DTYPE, F32, integers  # noqa: E402


def share(n, other=1.0):
    """So that some 300 of n products are not 0."""
    return min(1.0, 300 / (n * other)) if other < 1 else min(1.0, (300 / n) ** 0.5)


def same(name, got, ref):
    """ref: the exact values in float64, below 2^24."""
    largest = ref.abs().max().item()
    assert got.shape == ref.shape and largest < 2 ** 24, (name, largest)
    want = ref.to(got.dtype)
    wrong = (got != want).sum().item()
    assert wrong == 0, (name, wrong, got.numel(), (got != want).nonzero()[:4].tolist())


def weight(gen, t, int8, d_in, d_out, n):
    """W, w_scale (powers of two) and the weight in float64, for sums over n."""
    if not int8:
        W = integers(gen, (d_out, d_in), 2, share(n), "cuda").to(DTYPE[t])
        return W, None, W.double()
    q = integers(gen, (d_out, d_in), 127, share(n), "cuda").to(torch.int8)
    scale = torch.exp2(torch.randint(-1, 3, (d_out,), generator=gen, device="cuda").float())
    return q, scale, q.double() * scale.double()[:, None]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[2:])) + "-" +
                         ("f32", "bf16")[c[0]] + ("-int8" if c[1] else ""))
def test_every_variant(case):
    t, int8, tokens, d_in, d_out = case
    print("   ", case, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(tokens + d_in + d_out)
    # some 300 products of at most top x 2, with codes top x 127 x 4: 2.5 million
    # at most, of the 16.7 million that float32 counts
    dt, top = DTYPE[t], 2 if t == BF16 else 15 if int8 else 4095
    x = integers(gen, (tokens, d_in), top, share(d_in), "cuda").to(dt)
    W, scale, W64 = weight(gen, t, int8, d_in, d_out, d_in)
    bias = integers(gen, (d_out,), 100, 1.0, "cuda").float()
    r = integers(gen, (tokens, d_out), 100, 1.0, "cuda").to(dt)
    x64 = x.double()
    u64 = x64 @ W64.t() + bias.double()
    y, u = dense_forward(x, W, bias, r, "relu", scale, save_u=True)
    same("u", u, u64)
    same("y", y, u64.clamp(min=0) + r.double())
    y, _ = dense_forward(x, W, w_scale=scale)
    same("y of x W^T", y, u64 - bias.double())
    del u64, y, u

    g_share = share(d_out)
    g_y = integers(gen, (tokens, d_out), top, g_share, "cuda").to(dt)
    W, scale, W64 = weight(gen, t, int8, d_in, d_out, d_out)
    x = integers(gen, (tokens, d_in), 2, share(tokens, g_share), "cuda").to(dt)
    u = integers(gen, (tokens, d_out), 1, 1.0, "cuda").to(dt)
    for act in ("none", "relu"):
        g_u = g_y.double() if act == "none" else g_y.double() * (u > 0)
        ref = g_u @ W64
        g_x, none, g_b = dense_backward(g_y, W, u=u, activation=act, w_scale=scale, need_g_bias=True)
        same(act + " g_x alone", g_x, ref)
        assert none is None and torch.equal(g_b, g_u.sum(0).float())
        if int8:
            continue
        ref_W = g_u.t() @ x.double()
        _, g_W, _ = dense_backward(g_y, W, x, u, act, need_g_x=False, need_g_W=True)
        same(act + " g_W alone", g_W, ref_W)
        g_x, g_W, g_b = dense_backward(g_y, W, x, u, act, need_g_W=True, need_g_bias=True)
        same(act + " g_x", g_x, ref)
        same(act + " g_W", g_W, ref_W)
        assert torch.equal(g_b, g_u.sum(0).float())


def filled(gen, shape, top, part, dtype, rows=65_536):
    """integers() into a large tensor, some rows at a time."""
    out = torch.empty(shape, device="cuda", dtype=dtype)
    for i in range(0, shape[0], rows):
        n = min(rows, shape[0] - i)
        out[i:i + n] = integers(gen, (n, shape[1]), top, part, "cuda")
    return out


@pytest.mark.parametrize("t", [BF16, F32], ids=["bf16", "f32"])
def test_rows_past_32_bits(t):
    """y, u, residual, g_y and g_u of more than 2^32 elements each; every
    element of every output."""
    tokens, d_in, d_out = 300_031, 64, 14_336
    assert tokens * d_out > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(16)
    dt = DTYPE[t]
    x = integers(gen, (tokens, d_in), 2, 0.05, "cuda").to(dt)
    W = integers(gen, (d_out, d_in), 2, 0.2, "cuda").to(dt)
    bias = integers(gen, (d_out,), 3, 1.0, "cuda").float()
    r = filled(gen, (tokens, d_out), 3, 0.1, dt)
    y, u = dense_forward(x, W, bias, r, "relu", save_u=True)
    W64, b64 = W.double(), bias.double()
    for i in range(0, tokens, 10_000):
        u64 = x[i:i + 10_000].double() @ W64.t() + b64
        same("u", u[i:i + 10_000], u64)
        same("y", y[i:i + 10_000], u64.clamp_(min=0) + r[i:i + 10_000].double())
    del y
    g_x, g_W, g_b = dense_backward(r, W, x, u, "relu", need_g_W=True, need_g_bias=True)
    ref = torch.zeros(d_out, d_in, device="cuda", dtype=torch.float64)
    sums = ref.new_zeros(d_out)
    for i in range(0, tokens, 10_000):
        g_u = (u[i:i + 10_000] > 0) * r[i:i + 10_000].double()
        same("g_x", g_x[i:i + 10_000], g_u @ W64)
        ref += g_u.t() @ x[i:i + 10_000].double()
        sums += g_u.sum(0)
    same("g_W", g_W, ref)
    same("g_bias", g_b, sums)
    # (the sums show single lost ranges: most of them are of hundreds)
    assert ref.abs().mean() > 20 and sums.abs().mean() > 100


@pytest.mark.parametrize("tokens", [3, 40, 300])
@pytest.mark.parametrize("int8", [0, 1], ids=["bf16", "int8"])
def test_weights_past_32_bits(int8, tokens):
    """W (and g_W, INT8 codes and their widened copy) of more than 2^32
    elements; every element of every output."""
    d_in, d_out = 4096, 1_048_584
    assert d_in * d_out > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(17)
    x = integers(gen, (tokens, d_in), 2, 0.25, "cuda").bfloat16()
    bias = integers(gen, (d_out,), 100, 1.0, "cuda").float()
    scale = None
    if int8:
        W = filled(gen, (d_out, d_in), 127, 0.25, torch.int8)
        scale = torch.exp2(torch.randint(-1, 3, (d_out,), generator=gen, device="cuda").float())
    else:
        W = filled(gen, (d_out, d_in), 2, 0.25, torch.bfloat16)
    g_y = filled(gen, (d_out, tokens), 2, 0.02, torch.bfloat16).t().contiguous()
    y, _ = dense_forward(x, W, bias, w_scale=scale)
    g_x, g_W, g_b = dense_backward(g_y, W, x, w_scale=scale, need_g_W=not int8, need_g_bias=True)
    ref = torch.zeros(tokens, d_in, device="cuda", dtype=torch.float64)
    for i in range(0, d_out, 65_536):
        at = slice(i, min(d_out, i + 65_536))
        w64 = W[at].double()
        if int8:
            w64 *= scale[at].double()[:, None]
        same("y", y[:, at], x.double() @ w64.t() + bias[at].double())
        ref += g_y[:, at].double() @ w64
        if not int8:
            same("g_W", g_W[at], g_y[:, at].double().t() @ x.double())
    same("g_x", g_x, ref)
    same("g_bias", g_b, g_y.double().sum(0))
    assert ref.abs().mean() > 50


@pytest.mark.parametrize("t,tokens,width", [(F32, (1 << 30) - 64, 4), (BF16, 1 << 30, 8)],
                         ids=["f32", "bf16"])
def test_most_rows(t, tokens, width):
    """The most rows that the calls take (float32: 2^24 - 1 tiles): every element
    of every output. (Sums of 2^30 products of -1, 0 and 1 stay some ten
    thousand, whole numbers that float32 holds, in any order.)"""
    gen = torch.Generator(device="cuda").manual_seed(18)
    dt, part = DTYPE[t], 1 << 23
    x = filled(gen, (tokens, width), 1, 0.3, dt, part)
    g_y = filled(gen, (tokens, width), 1, 0.3, dt, part)
    W = integers(gen, (width, width), 2, 0.8, "cuda").to(dt)
    bias = integers(gen, (width,), 1, 1.0, "cuda").float()
    y, u = dense_forward(x, W, bias, g_y, "relu", save_u=True)
    g_x, g_W, g_b = dense_backward(g_y, W, x, u, "relu", need_g_W=True, need_g_bias=True)
    W64, b64 = W.double(), bias.double()
    ref = torch.zeros(width, width, device="cuda", dtype=torch.float64)
    sums = ref.new_zeros(width)
    for i in range(0, tokens, part):
        at = slice(i, min(tokens, i + part))
        x64, g64 = x[at].double(), g_y[at].double()
        u64 = x64 @ W64.t() + b64
        same("u", u[at], u64)
        same("y", y[at], u64.clamp(min=0) + g64)
        g64 *= u64 > 0
        same("g_x", g_x[at], g64 @ W64)
        # (column by column: a product of so few outputs is slow in the library)
        ref += torch.stack([(g64 * x64[:, j:j + 1]).sum(0) for j in range(width)], 1)
        sums += g64.sum(0)
        if i % (16 * part) == 0:
            print("    row", i, flush=True)
    same("g_W", g_W, ref)
    same("g_bias", g_b, sums)

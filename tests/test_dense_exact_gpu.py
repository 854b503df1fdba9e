"""The dense linear on operands of small integers, bit for bit: every product
and sum is exact in float32 in any order, so an output is the exact value
rounded once to its type, on every kernel variant that the plans choose
(dense_cases.py)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here is gpu-marked
    pytest.skip("no GPU", allow_module_level=True)

from orthogonal_equivalence_amd.dense import dense_backward, dense_forward  # noqa: E402
from tests.dense_cases import BF16, CASES, DTYPE, integers  # noqa: E402


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

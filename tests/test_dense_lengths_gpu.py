"""Reductions of every number of steps, whole and cut, bit for bit on integer
operands: the first and last steps of the kernels' rings, where copies, waits
and zeroed tails differ from the steady state."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here is gpu-marked
    pytest.skip("no GPU", allow_module_level=True)

from orthogonal_equivalence_amd.dense import dense_backward, dense_forward  # noqa: E402
from tests.dense_cases import BF16, DTYPE, F32, integers, operands  # noqa: E402

KINDS = [(F32, 0), (BF16, 0), (BF16, 1)]
IDS = ["f32", "bf16", "int8"]


def same(got, ref, what):
    assert ref.abs().max() < 2 ** 24, what
    assert torch.equal(got, ref.to(got.dtype)), what


def forward(gen, t, int8, tokens, d_in, d_out):
    x, W = operands(gen, t, d_in, (tokens, d_in), (d_out, d_in), "cuda")
    scale, W64 = None, W.double()
    if int8:
        W = integers(gen, (d_out, d_in), 20, 0.5, "cuda").to(torch.int8)
        scale = torch.exp2(torch.randint(-1, 3, (d_out,), generator=gen, device="cuda").float())
        W64 = W.double() * scale.double()[:, None]
    y, u = dense_forward(x, W, w_scale=scale, save_u=True)
    ref = x.double() @ W64.t()
    same(y, ref, (t, int8, tokens, d_in, d_out))
    assert torch.equal(u, y)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("tokens", range(1, 9))
def test_few_tokens(kind, tokens):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    for d_in in [*range(8, 1400, 8 * 11), *range(1000, 9000, 8 * 101), *range(16, 4200, 16 * 23)]:
        forward(gen, *kind, tokens, d_in, 40)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("tokens,d_out", [(20, 72), (200, 328), (700, 1544), (700, 4104)])
def test_every_number_of_steps(kind, tokens, d_out):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    step = 32 if kind[0] == F32 else 64
    for n in range(1, 24):  # whole steps, one vector less, one more
        for d_in in (n * step - 8, n * step, n * step + 8):
            if d_in > 0:
                forward(gen, *kind, tokens, d_in, d_out)


@pytest.mark.parametrize("int8", [0, 1], ids=["bf16", "int8"])
@pytest.mark.parametrize("tokens,d_out", [(1030, 9096), (1030, 9216), (4100, 8200)])
def test_large_tiles(int8, tokens, d_out):
    """256 x 256 tiles, one and several a workgroup."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    for d_in in range(32, 32 * 24, 32):
        forward(gen, BF16, int8, tokens, d_in, d_out)


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d_in,d_out", [(40, 72), (328, 264), (4104, 136)])
def test_weight_gradient_of_every_number_of_tokens(t, d_in, d_out):
    gen = torch.Generator(device="cuda").manual_seed(d_in)
    W = torch.zeros(d_out, d_in, device="cuda", dtype=DTYPE[t])
    for tokens in [*range(1, 140), *range(140, 1500, 37)]:
        g_y, x = operands(gen, t, tokens, (d_out, tokens), (d_in, tokens), "cuda")
        g_y, x = g_y.t().contiguous(), x.t().contiguous()
        u = integers(gen, (tokens, d_out), 1, 1.0, "cuda").to(DTYPE[t])
        g_u = g_y.double() * (u > 0)
        ref = g_u.t() @ x.double()
        for need_g_x in (False, True):
            g_x, g_W, g_b = dense_backward(g_y, W, x, u, "relu", need_g_x=need_g_x, need_g_W=True,
                                           need_g_bias=True)
            same(g_W, ref, (t, tokens, d_in, d_out, need_g_x))
            assert torch.equal(g_b, g_u.sum(0).float()), (tokens, d_out)
            assert g_x is None or not g_x.any()


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("tokens,d_in", [(5, 40), (100, 328), (700, 1544), (4100, 8200)])
def test_input_gradient_of_every_number_of_steps(kind, tokens, d_in):
    t, int8 = kind
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    step = 32 if t == F32 else 64
    for n in range(1, 24, 4 if tokens == 4100 else 1):
        for d_out in (n * step - 8, n * step, n * step + 8):
            g_y, W = operands(gen, t, d_out, (tokens, d_out), (d_in, d_out), "cuda")
            W = W.t().contiguous()
            scale, W64 = None, W.double()
            if int8:
                W = W.to(torch.int8)
                scale = torch.exp2(torch.randint(-1, 3, (d_out,), generator=gen,
                                                 device="cuda").float())
                W64 = W64 * scale.double()[:, None]
            g_x, _, _ = dense_backward(g_y, W, w_scale=scale)
            same(g_x, g_y.double() @ W64, (kind, tokens, d_in, d_out))

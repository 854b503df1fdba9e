"""The activations and their slopes in float32 storage, on intervals, against
float64: the root mean square of the error over that of the value, in half
steps of float32 (2^-24).

Bounds: expf and erfcf within one step (two half steps: 1.15 root mean square),
every other operation half a step (0.58), each weighted with what the value
does with it (below, as its share of the value's root mean square), and a
constant's rounding counted with its product. In order of the formula:
  gelu       u * 1/sqrt 2 (0.77, times |u| phi / Phi: 1.5 at most on [-1, 0],
             0.3 above), erfcf 1.15, the product 0.58
  silu       expf (and e^-u's share of 1 + e^-u), the sum, the quotient
  gelu_tanh  the argument (three operations and a constant, 1.2, times the
             argument: at most 1.8 on [-1, 0], where the logistic function
             passes on half and more), then as silu
and the slopes' second terms, u phi or u p (1 - p) 2 z', of at most 0.6 of the
value and four further operations."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here is gpu-marked
    pytest.skip("no GPU", allow_module_level=True)

from orthogonal_equivalence_amd.dense import dense_backward, dense_forward  # noqa: E402


def act64(u, name):
    """act(u) and its slope in float64."""
    if name == "gelu":
        cdf = torch.special.ndtr(u)
        return u * cdf, cdf + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    c, a = (math.sqrt(2 / math.pi), 0.044715) if name == "gelu_tanh" else (0.5, 0.0)
    p = torch.special.expit(2 * c * (u + a * u ** 3))
    q = torch.special.expit(-2 * c * (u + a * u ** 3))
    return u * p, p + u * p * q * 2 * c * (1 + 3 * a * u * u)


def off(got, ref):
    assert torch.isfinite(got).all()
    return ((got.double() - ref).square().mean() / ref.square().mean()).sqrt().item() * 2 ** 24


# activation, interval, bound of the value, bound of the slope
BOUNDS = [("gelu", -1.0, 0.0, 2.0, 2.5), ("gelu", 0.0, 1.0, 1.4, 1.4), ("gelu", -3.0, 3.0, 1.4, 1.4),
          ("gelu", 3.0, 8.0, 1.4, 1.4), ("silu", -1.0, 0.0, 1.5, 1.75), ("silu", 0.0, 1.0, 1.5, 1.75),
          ("silu", -8.0, -3.0, 1.5, 2.0), ("silu", 3.0, 8.0, 1.5, 1.5),
          ("gelu_tanh", -1.0, 0.0, 2.0, 2.5), ("gelu_tanh", 0.0, 1.0, 1.5, 1.5),
          ("gelu_tanh", 3.0, 8.0, 1.5, 1.5)]


@pytest.mark.parametrize("tokens", [1, 40], ids=["few", "tiles"])
@pytest.mark.parametrize("name,lo,hi,value,slope", BOUNDS)
def test_float32_activation(name, lo, hi, value, slope, tokens):
    n = 65_536
    u = torch.linspace(lo, hi, n, device="cuda")
    x, W = torch.zeros(tokens, 8, device="cuda"), torch.zeros(n, 8, device="cuda")
    y, kept = dense_forward(x, W, u, activation=name, save_u=True)  # u = bias
    assert torch.equal(kept, u.expand(tokens, -1)) and torch.equal(y, y[:1].expand(tokens, -1))
    g_y = torch.zeros(tokens, n, device="cuda")
    g_y[tokens - 1] = 1.0
    _, _, g_b = dense_backward(g_y, W, u=kept, activation=name, need_g_x=False, need_g_bias=True)
    y64, slope64 = act64(u.double(), name)
    v, s = off(y[0], y64), off(g_b, slope64)
    print(f"    {name} [{lo}, {hi}]: value {v:.2f} ({value}), slope {s:.2f} ({slope})", flush=True)
    assert v <= value and s <= slope

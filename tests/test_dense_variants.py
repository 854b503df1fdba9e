"""The cases of dense_cases.py (CPU): they reach every kernel variant that the
dense linear's plans choose for drawn sizes, and their operands show a lost
step, split or range of a sum, an index that wraps, and shortened operands."""
import math
import random

import pytest

torch = pytest.importorskip("torch")

from tests.dense_cases import BF16, CASES, DTYPE, F32, integers, operands, variants  # noqa: E402
from tests.test_dense_plan import plans  # noqa: E402


def test_cases_reach_every_variant():
    rng = random.Random(11)

    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    drawn = []
    for _ in range(30_000):
        step = rng.choice((8, 8, 16, 256))
        d_in, d_out = (max(step, size(8, 14336) // step * step) for _ in range(2))
        drawn.append((rng.choice((F32, BF16, BF16)), int(rng.random() < 0.3), size(1, 8192), d_in,
                      d_out))
    reached = set()
    for c, p in zip(CASES, plans(CASES)):
        reached |= variants(c, p)
    missed = {}
    for c, p in zip(drawn, plans(drawn)):
        for v in variants(c, p) - reached:
            missed.setdefault(v, c)
    assert not missed, missed
    assert len(reached) > 100


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n", [64, 4096, 14_336, 300_031, 1_048_584])
def test_operands_show_lost_products(t, n):
    """Sums are whole numbers below 2^24; with 32 consecutive products lost, a
    split's part lost, an index off by 2^32 bytes' worth or operands cut to
    bfloat16 (float32) most of a row's sums change, and none are zero all
    over."""
    gen = torch.Generator().manual_seed(n)
    a, b = operands(gen, t, n, (4, n), (32, n), "cpu")
    a64, b64 = a.double(), b.double()
    ref = a64 @ b64.t()
    assert (a64.abs() @ b64.abs().t()).max() < 2 ** 24
    out = ref.to(DTYPE[t])
    assert (out != 0).double().mean() > 0.9
    part = max(32, n // 16 // 32 * 32)
    lost = [slice(n - part, n), slice(n // 2, n // 2 + part)]
    if n <= 14_336:  # (a step of so few of the products has some that are not 0)
        lost.append(slice(n - 32, n))
    for s in lost:
        keep = a64.clone()
        keep[:, s] = 0
        changed = ((keep @ b64.t()).to(DTYPE[t]) != out).double().mean()
        assert changed > (0.9 if s.stop - s.start > 0.05 * n else 0.2), (s, changed)
    shifted = torch.roll(b64, 8, dims=1)
    assert ((a64 @ shifted.t()).to(DTYPE[t]) != out).double().mean() > 0.9
    if t == F32:
        assert ((a.bfloat16().double() @ b64.t()).to(DTYPE[t]) != out).double().mean() > 0.9


def test_integers():
    v = integers(torch.Generator().manual_seed(1), (1000, 1000), 3, 0.25, "cpu").float()
    assert v.abs().max() == 3 and abs((v != 0).float().mean() - 0.25) < 0.01 and abs(v.mean()) < 0.01

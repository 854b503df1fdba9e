"""The sizes of vocab_routes.py take the kernels that their names say (CPU)."""
import pytest

from tests.test_vocab_plan import plans
from tests.vocab_routes import RANGES, ROUTES, SORTED

# of the forward and of the backward of both gradients: columns on 256 x 256
# tiles, whether the backward runs on them, g_W on the kernel for few tokens, pieces
EXPECTED = {
    "tiles, float32": (0, 0, 0, 1),
    "tiles": (0, 0, 0, 1),
    "few tokens, float32": (0, 0, 1, 1),
    "few tokens": (0, 0, 1, 1),
    "rows padded to a tile": (0, 1, 0, 1),
    "256 x 256 tiles, last panel padded": (26351, 1, 0, 1),
    "256 x 256 tiles, last columns on small tiles": (65536, 1, 0, 1),
    "256 x 256 tiles, two pieces": (131072, 1, 0, 2),
}


@pytest.mark.parametrize("name", ROUTES)
def test_route(name):
    case = ROUTES[name]
    p, = plans([(*case, 0)])
    assert (p["dense"], p["b_dense"], p["few"], len(p["pieces"])) == EXPECTED[name]
    if p["b_dense"]:  # (g_x's reduction in ranges, summed from slabs)
        assert p["splits"] > 1 and p["padded"] % 256 == 0
        assert p["pieces"][0]["dense"] == min(p["dense"] or case[3], p["piece"])


@pytest.mark.parametrize("name", SORTED)
def test_sorted_route(name):
    p, = plans([SORTED[name]])
    dense = {"sorted, 256 x 256 tiles": 20000, "sorted, both": 49152}.get(name, 0)
    assert p["cells"] and p["dense"] == dense


@pytest.mark.parametrize("name", RANGES)
def test_ranges(name):
    _, tokens, _, vocab, top = RANGES[name]
    p, = plans([RANGES[name]])
    assert p["cells"] == (top > 0) and 0 < tokens % p["rows"] < 256 and p["rows"] < tokens
    # (16384 cells a row of cells, the most that are sorted)
    assert p["dense"] == (vocab if top else (vocab // 256) * 256)

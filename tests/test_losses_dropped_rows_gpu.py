"""Rows that add nothing to a gradient, whatever their x holds, by every route of
the losses' backward (GPU)."""
import math

import pytest
import torch

from tests import vocab_cases as V
from tests.vocab_routes import DTYPE, ROUTES

pytestmark = pytest.mark.gpu

L = pytest.importorskip("orthogonal_equivalence_amd.losses",
                        reason="libpoetx.so not built (run the build first)")


def _dirty(x, rows):
    """x with NaN, infinities and the largest values in `rows`, and with zeros there."""
    d = x.shape[1]
    bad = torch.tensor([math.nan, math.inf, -math.inf, 3e38], device="cuda").repeat(d // 4)
    clean = torch.where(rows[:, None], torch.zeros_like(x), x)
    return clean, torch.where(rows[:, None], bad.to(x.dtype), x)


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("name", ROUTES)
def test_rows_without_gradient(name):
    """Rows weighted by 0 (a padded batch whose targets are not masked): no part of
    their x reaches g_W, and their g_x is 0, at any number of tokens."""
    print("weights of 0", name, flush=True)
    t, tokens, d, vocab = ROUTES[name]
    x, W = V.inputs(tokens, d, vocab, DTYPE[t], 1, True)
    targets = V.draw_targets(tokens, vocab, 2)
    ids, teacher = V.draw_teacher(tokens, vocab, 6, 3)
    off = torch.rand(tokens, generator=torch.Generator().manual_seed(4)).cuda() < 0.3
    off[3] = True
    g = torch.where(off, 0.0, 1.0)
    clean, dirty = _dirty(x, off)
    loss, lse = L.cross_entropy_forward(clean, W, targets)
    _, kd_lse, z = L.distill_forward(clean, W, ids, teacher, 2.0)
    nan = torch.full((), math.nan, device="cuda")
    out = []
    for v in (clean, dirty):
        # (what the forward leaves for such rows may be NaN too)
        bad = v is dirty
        own = torch.where(off, nan, lse) if bad else lse
        kd_own = torch.where(off, nan, kd_lse) if bad else kd_lse
        z_own = torch.where(off[:, None], nan, z) if bad else z
        out.append((*L.cross_entropy_backward(g, v, W, targets, own, need_g_W=True),
                    *L.cross_entropy_backward(g, v, W, targets, own, g_lse=-0.5 * g, need_g_W=True),
                    *L.distill_backward(g, v, W, ids, teacher, kd_own, z_own, 2.0, need_g_W=True)))
    assert _same(*out)
    for g_x in out[1][::2]:
        assert bool((g_x[off] == 0).all())

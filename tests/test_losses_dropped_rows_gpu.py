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


@pytest.mark.parametrize("name", ROUTES)
def test_rows_that_take_no_part(name):
    """Padding may hold anything: NaN and infinities in the x of a row without a target or
    entries reach no other row's results and no gradient."""
    print("no part", name, flush=True)
    t, tokens, d, vocab = ROUTES[name]
    x, W = V.inputs(tokens, d, vocab, DTYPE[t], 1, True)
    targets = V.draw_targets(tokens, vocab, 2, ignored=0.4)
    ids, teacher = V.draw_teacher(tokens, vocab, 6, 3)
    ids = torch.where((targets < 0)[:, None], -1, ids)
    g = torch.rand(tokens, generator=torch.Generator().manual_seed(5)).cuda() + 0.5
    rows = targets < 0
    held = (ids >= 0) & (teacher > -math.inf)
    kd_rows = ~held.any(1)
    out = []
    for v, kd in zip(_dirty(x, rows), _dirty(x, kd_rows)):
        loss, lse = L.cross_entropy_forward(v, W, targets)
        got = [loss, lse, *L.cross_entropy_backward(g, v, W, targets, lse, g_lse=g, need_g_W=True),
               *L.cross_entropy_backward(g, v, W, targets, lse)[:1]]
        assert all(bool((r[rows] == 0).all()) for r in (got[0], got[1], got[2], got[4]))
        loss, lse, z = L.distill_forward(kd, W, ids, teacher, 2.0)
        got += [loss, lse, *L.distill_backward(g, kd, W, ids, teacher, lse, z, 2.0, need_g_W=True)]
        assert all(bool((r[kd_rows] == 0).all()) for r in got[5:8])
        # (masked by the teacher's logits alone: entries with ids)
        own = torch.where(ids < 0, 7, ids)
        masked = torch.where(ids < 0, -math.inf, teacher)
        loss, lse, z = L.distill_forward(kd, W, own, masked, 2.0)
        got += [loss, lse, *L.distill_backward(g, kd, W, own, masked, lse, z, 2.0, need_g_W=True)]
        out.append(got)
        assert all(bool(torch.isfinite(r).all()) for r in got)
    assert _same(*out)


@pytest.mark.parametrize("name", ROUTES)
def test_ids_past_the_vocabulary(name):
    """Read nowhere: the row's loss and g_x are NaN and g_W is; the other rows keep their
    bits."""
    print("past the vocabulary", name, flush=True)
    t, tokens, d, vocab = ROUTES[name]
    x, W = V.inputs(tokens, d, vocab, DTYPE[t], 1, True)
    targets = V.draw_targets(tokens, vocab, 2)
    ids, teacher = V.draw_teacher(tokens, vocab, 6, 3)
    g = torch.ones(tokens, device="cuda")
    row = tokens - 2
    targets[row] = ids[row, 0] = 5
    teacher[row, 0] = 0.5

    def both(targets, ids):
        loss, lse = L.cross_entropy_forward(x, W, targets)
        first = [loss, lse, *L.cross_entropy_backward(g, x, W, targets, lse, need_g_W=True)]
        loss, lse, z = L.distill_forward(x, W, ids, teacher, 2.0)
        return first + [loss, lse, *L.distill_backward(g, x, W, ids, teacher, lse, z, 2.0,
                                                       need_g_W=True)]

    ref = both(targets, ids)
    keep = torch.arange(tokens, device="cuda") != row
    for bad in (vocab, vocab + 255, 2 ** 31 + 5, 2 ** 40):
        targets[row] = ids[row, 0] = bad
        got = both(targets, ids)
        for k in (0, 2, 4, 6):
            assert torch.equal(got[k][keep], ref[k][keep]) and bool(torch.isnan(got[k][row]).all())
        for k in (3, 7):
            assert bool(torch.isnan(got[k]).all())
        for k in (1, 5):
            assert torch.equal(got[k], ref[k])

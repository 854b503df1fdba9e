"""bf16 gradients of fewer than 256 tokens (GPU): as exact as float32 g_z gives them,
one rounding of the result. (With g_z rounded to bf16 once, its largest entry's
rounding shifts a whole row by up to half a step more.)"""
import math

import pytest
import torch

from tests import test_losses_gpu as G
from tests import vocab_cases as V

pytestmark = pytest.mark.gpu

L = pytest.importorskip("orthogonal_equivalence_amd.losses",
                        reason="libpoetx.so not built (run the build first)")

SIZES = [  # tokens, d, vocab
    (1, 8, 5), (1, 256, 1000), (2, 1280, 6400), (5, 72, 3001), (17, 200, 257), (31, 2048, 9001),
    (33, 264, 2049), (64, 512, 9001), (97, 1280, 28160), (128, 256, 20000), (128, 4096, 3001),
    # (256 x 256 tiles: rows of both parts by sixteens, the last ones ragged)
    (129, 256, 110749), (144, 1024, 41256), (166, 768, 41256), (240, 544, 66539), (255, 256, 100096),
    (200, 1024, 5000), (255, 72, 7001),
]


def tolerances(ref, x, W, temperature, part, listed):
    """What float32 loses (test_losses_gpu.py), what the two parts of g_z leave of it (a part
    below 2^-16 of the first, and 2^-8 of the second, below 2^-8 of the first), and half
    a step of the result."""
    tol_x, tol_W = G.gradient_tolerances(ref, x, W, "f32", temperature, part, listed)
    xs = torch.where(part[:, None], x.double(), torch.zeros_like(x.double())).abs()
    left = (2.0 ** -16 + 2.0 ** -24) * ref["g_z"].abs()
    tol_x = tol_x + left.mm(W.double().abs()) + 2.0 ** -8 * ref["g_x"].abs()
    tol_W = tol_W + left.t().mm(xs) + 2.0 ** -8 * ref["g_W"].abs()
    return tol_x * (1 + 2.0 ** -7), tol_W * (1 + 2.0 ** -7)


# (several pieces of the vocabulary: on small tiles, with g_W's own kernel, on 256 x 256 tiles)
PIECES = [(200, 64, 1_500_000), (100, 64, 3_000_001), (255, 256, 1_100_000)]


@pytest.mark.parametrize("tokens,d,vocab", SIZES + PIECES)
def test_cross_entropy(tokens, d, vocab):
    print(f"few tokens {tokens} {d} {vocab}", flush=True)
    x, W = V.inputs(tokens, d, vocab, "bf16", 21, True)
    t = V.draw_targets(tokens, vocab, 22)
    gen = torch.Generator().manual_seed(23)
    g = (torch.rand(tokens, generator=gen) + 0.5).cuda()
    _, lse = L.cross_entropy_forward(x, W, t)
    part = t >= 0
    for g_lse in (None, torch.randn(tokens, generator=gen).cuda()):
        ref = V.targets_reference(x, W, t, g_loss=g, g_lse=g_lse, lse=lse)
        a = g if g_lse is None else g + g_lse
        G.magnitudes(ref, g, a, 1.0, part, t[:, None], part.double()[:, None], lse, True, x, W)
        tol_x, tol_W = tolerances(ref, x, W, 1.0, part, 1)
        g_x, g_W = L.cross_entropy_backward(g, x, W, t, lse, g_lse=g_lse, need_g_W=True)
        G.within("g_x", g_x, ref["g_x"], tol_x)
        G.within("g_W", g_W, ref["g_W"], tol_W)
        only, _ = L.cross_entropy_backward(g, x, W, t, lse, g_lse=g_lse)
        G.within("g_x alone", only, ref["g_x"], tol_x)
        _, only = L.cross_entropy_backward(g, x, W, t, lse, g_lse=g_lse, need_g_x=False,
                                           need_g_W=True)
        G.within("g_W alone", only, ref["g_W"], tol_W)


@pytest.mark.parametrize("tokens,d,vocab", SIZES)
def test_distill(tokens, d, vocab):
    print(f"few tokens, lists {tokens} {d} {vocab}", flush=True)
    temperature, top = 2.0, min(vocab, 7)
    x, W = V.inputs(tokens, d, vocab, "bf16", 31, True)
    ids, teacher = V.draw_teacher(tokens, vocab, top, 32)
    g = (torch.rand(tokens, generator=torch.Generator().manual_seed(33)) + 0.5).cuda()
    _, lse, z = L.distill_forward(x, W, ids, teacher, temperature)
    ref = V.teacher_reference(x, W, ids, teacher, temperature, g_loss=g, lse=lse)
    held = (ids >= 0) & (teacher > -math.inf)
    part = held.any(1)
    t64 = torch.where(held, teacher.double() / temperature, -math.inf)
    p = torch.where(part[:, None], torch.softmax(t64, 1), torch.zeros_like(t64)).nan_to_num(0.0)
    G.magnitudes(ref, g, g * temperature, temperature, part, ids, p, lse, True, x, W)
    tol_x, tol_W = tolerances(ref, x, W, temperature, part, top + 64)
    g_x, g_W = L.distill_backward(g, x, W, ids, teacher, lse, z, temperature, need_g_W=True)
    G.within("g_x", g_x, ref["g_x"], tol_x)
    G.within("g_W", g_W, ref["g_W"], tol_W)
    only, _ = L.distill_backward(g, x, W, ids, teacher, lse, z, temperature)
    G.within("g_x alone", only, ref["g_x"], tol_x)


@pytest.mark.parametrize("tokens,d,vocab", [(7, 512, 3001), (200, 512, 40001)])
def test_infinite_weights_stay_infinite(tokens, d, vocab):
    """A g_z past bf16's range has no second part: infinities, not NaN, in its row."""
    x, W = V.inputs(tokens, d, vocab, "bf16", 41, True)
    x[:, 0], W[:, 0] = 1, 1
    t = V.draw_targets(tokens, vocab, 42, ignored=0)
    t[3] = 5
    g = torch.ones(tokens, device="cuda")
    g[3] = 3.4e38
    _, lse = L.cross_entropy_forward(x, W, t)
    g_x, g_W = L.cross_entropy_backward(g, x, W, t, lse, need_g_W=True)
    assert g_W[5, 0].item() == -math.inf
    keep = torch.arange(tokens, device="cuda") != 3
    assert bool(torch.isfinite(g_x[keep]).all())

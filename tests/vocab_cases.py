"""Inputs and the float64 reference of the losses over a vocabulary (test
helpers, shared by the test_losses_*.py files)."""
from __future__ import annotations

import math

import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# half a step of a rounding, relative to the value
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def reference(x, W, ids, p, part, log_p, temperature=1.0, g_loss=None, g_lse=None, lse=None):
    """Everything in float64 from the definitions. ids [tokens, top] with p and
    log_p [tokens, top] (0 where an entry takes no part), part [tokens]. Forward: loss, lse, z.
    With g_loss also g_z, g_x, g_W (from `lse`, the forward's, where given)."""
    x, W = x.double(), W.double()
    z = x.mm(W.t())
    held = (p != 0) & (ids >= 0)
    at = torch.where(ids >= 0, z.gather(1, ids.clamp(min=0)), torch.zeros_like(p))
    full = torch.logsumexp(z / temperature, 1)
    own = torch.where(part, full, torch.zeros_like(full))
    terms = torch.where(held, p * (log_p - at / temperature + own[:, None]), torch.zeros_like(p))
    out = {"loss": temperature ** 2 * terms.sum(1), "lse": own, "z": at, "logits": z}
    if g_loss is None:
        return out
    g = torch.where(part, g_loss.double(), torch.zeros_like(own)) * temperature
    a = g if g_lse is None else torch.where(part, g + g_lse.double(), torch.zeros_like(g))
    lse = own if lse is None else lse.double()
    g_z = torch.exp(z / temperature - lse[:, None]) * a[:, None]
    g_z = torch.where(part[:, None], g_z, torch.zeros_like(g_z))
    g_z.scatter_add_(1, ids.clamp(min=0), torch.where(held, -g[:, None] * p, torch.zeros_like(p)))
    xs = torch.where(part[:, None], x, torch.zeros_like(x))
    return dict(out, g_z=g_z, g_x=g_z.mm(W), g_W=g_z.t().mm(xs))


def targets_reference(x, W, targets, **kw):
    part = targets >= 0
    p = part.double()[:, None]
    return reference(x, W, targets[:, None], p, part, torch.zeros_like(p), **kw)


def teacher_reference(x, W, ids, teacher, temperature, **kw):
    t = teacher.double()
    held = (ids >= 0) & (t > -math.inf)
    part = held.any(1)
    t = torch.where(held, t / temperature, torch.full_like(t, -math.inf))
    top = torch.where(part, t.max(1).values, torch.zeros_like(t[:, 0]))
    e = torch.exp(t - top[:, None])
    total = torch.where(part, e.sum(1), torch.ones_like(top))
    log_p = torch.where(held, t - top[:, None] - torch.log(total)[:, None], torch.zeros_like(t))
    return reference(x, W, ids, e / total[:, None], part, log_p, temperature, **kw)


def inputs(tokens, d, vocab, dtype, seed, dyadic=False, device="cuda"):
    """x and W; with dyadic every logit is exact in float32 (x in {-1, 0, 1}, W
    multiples of 1/8), of standard deviation about 2."""
    gen = torch.Generator().manual_seed(seed)
    if dyadic:
        x = torch.randint(-1, 2, (tokens, d), generator=gen).float()
        most = max(1, round(40 / math.sqrt(d)))
        W = torch.randint(-most, most + 1, (vocab, d), generator=gen).float() / 8
    else:
        x = torch.randn(tokens, d, generator=gen)
        W = torch.randn(vocab, d, generator=gen) * (2 / math.sqrt(d))
    return x.to(device, DT[dtype]), W.to(device, DT[dtype])


def draw_targets(tokens, vocab, seed, ignored=0.25, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    t = torch.randint(0, vocab, (tokens,), generator=gen)
    t[torch.rand(tokens, generator=gen) < ignored] = -100
    t[0] = vocab - 1
    if tokens > 2:
        t[1], t[2] = 0, -1
    return t.to(device)


def draw_teacher(tokens, vocab, top, seed, dtype="f32", device="cuda"):
    """Ids (some listed twice, some entries and whole rows absent) and logits
    (some -inf)."""
    gen = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, vocab, (tokens, top), generator=gen)
    if top > 1:
        ids[::3, 1] = ids[::3, 0]
    t = (3 * torch.randn(tokens, top, generator=gen)).to(DT[dtype])
    gone = torch.rand(tokens, top, generator=gen) < 0.2
    gone[1::5] = True
    gone[0] = False
    t[torch.rand(tokens, top, generator=gen) < 0.1] = -math.inf
    ids[gone] = -1
    t[0] = torch.where(torch.isinf(t[0]), torch.zeros_like(t[0]), t[0])
    ids[0, 0] = vocab - 1
    return ids.to(device), t.to(device)


def lse_tolerance(ref, temperature, d, x, W, dyadic):
    """What float32 may lose of lse, absolute, per row. The logits: sums of d
    products in any order, each step off by at most one step of float32 (exact
    when dyadic). The exponents c z - m: the constant, m and the difference each
    rounded, a half step of |c z| apiece. The sums of exponentials: chains of at
    most 64 columns in a lane, the tree, and vocab / 128 slots in a thread. The
    logarithm, its product with ln 2 and the sum, a step each of lse."""
    u = 2.0 ** -24
    z = ref["logits"].abs().max(1).values / temperature
    tol = u * (4 * z + 4 * ref["lse"].abs() + 128 + W.shape[0] / 128)
    if not dyadic:
        bound = x.double().abs().mm(W.double().abs().t()).max(1).values
        tol = tol + 2 * u * (d + 8) * bound / temperature
    return tol


F32, BF16 = 0, 1
# Sizes whose plans reach every kernel variant that drawn sizes do (held to it by
# test_vocab_plan.py). CASES: both directions of cross entropy; LISTED: of
# distillation, with the entries of a row's list.
CASES = [  # dtype, tokens, d, vocab
    (BF16, 65, 8, 11889), (BF16, 44, 8, 24458), (BF16, 1253, 8, 1), (BF16, 4834, 296, 1),
    (BF16, 471, 3712, 1), (BF16, 168, 336, 6449), (BF16, 16, 72, 96113), (F32, 1, 928, 15857),
    (BF16, 7398, 392, 279), (BF16, 1422, 8, 5376), (BF16, 5608, 256, 1106), (BF16, 585, 3584, 427),
    (BF16, 333, 448, 77312), (BF16, 42, 224, 129074), (BF16, 1189, 736, 15165), (F32, 40, 72, 63264),
    (F32, 20, 152, 74599), (BF16, 759, 768, 22239), (BF16, 5438, 80, 5913), (BF16, 2313, 2752, 1338),
    (BF16, 1056, 1312, 9504), (F32, 1, 1728, 45137), (F32, 631, 8, 65783), (F32, 39, 400, 40688),
    (BF16, 4, 2816, 49035), (BF16, 672, 2816, 9001), (BF16, 8100, 400, 5148), (BF16, 2560, 256, 14080),
    (BF16, 298, 256, 115906), (BF16, 650, 256, 69815), (BF16, 45, 1792, 88320), (F32, 4623, 8, 60672),
    (F32, 887, 1152, 1792), (F32, 84, 2048, 11439), (BF16, 1792, 1536, 14592), (F32, 23, 2048, 39497),
    (BF16, 3137, 2720, 3077), (F32, 7930, 96, 3471), (BF16, 3756, 3840, 2304), (BF16, 1350, 256, 109972),
    (F32, 4849, 16, 49508), (F32, 60, 2752, 30580), (F32, 1896, 1024, 2972), (BF16, 5600, 3392, 3840),
    (BF16, 2379, 320, 108458), (BF16, 4096, 2816, 36606), (BF16, 71, 208, 98288), (BF16, 73, 1024, 72448),
    (BF16, 101, 1792, 47872), (BF16, 153, 256, 110689), (BF16, 19, 3512, 115968),
    (BF16, 53, 1312, 119532),
]
# dtype, tokens, d, vocab, top
LISTED = [
    (BF16, 1, 8, 1, 6), (F32, 1, 8, 1, 29), (BF16, 4748, 3360, 6, 12),
    (F32, 2017, 256, 1, 92), (F32, 36, 8, 28221, 54), (BF16, 1792, 1528, 1, 71),
    (F32, 839, 8, 512, 23), (F32, 7122, 2624, 3, 2), (BF16, 138, 4064, 256, 1),
    (BF16, 274, 1024, 26351, 3), (BF16, 2, 192, 61450, 11), (BF16, 1263, 288, 14065, 85),
    (F32, 52, 72, 50853, 1), (BF16, 262, 256, 100366, 5), (BF16, 270, 2432, 10202, 4),
    (BF16, 953, 768, 17664, 16), (BF16, 6039, 512, 3401, 36), (BF16, 129, 3000, 17764, 10),
    (F32, 2482, 2336, 256, 1), (BF16, 399, 544, 66539, 10), (BF16, 4698, 8, 65522, 26),
    (F32, 35, 2816, 41863, 73), (BF16, 3606, 256, 70033, 25),
    (BF16, 68, 8, 118786, 2), (BF16, 97, 1280, 28160, 1), (BF16, 460, 1568, 46189, 2),
    (BF16, 1792, 256, 78091, 3), (BF16, 166, 768, 41256, 14), (BF16, 215, 256, 110749, 3),
]

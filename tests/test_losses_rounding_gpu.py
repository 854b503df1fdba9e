"""What the losses over a vocabulary round (GPU): the maximum and the sum of a
row's exponentials stay apart until the loss is formed, so a loss is off by
roundings of its own size, however large the logits are."""
import math

import pytest
import torch

from tests import vocab_cases as V
from tests.vocab_routes import DTYPE, ROUTES

pytestmark = pytest.mark.gpu

L = pytest.importorskip("orthogonal_equivalence_amd.losses",
                        reason="libpoetx.so not built (run the build first)")

U32 = 2.0 ** -24  # half a step of float32


def _inputs(case, offset):
    """Logits that are exact in float32 (multiples of 1/8 below 2^11), all of them
    `offset` higher by a column of their own."""
    t, tokens, d, vocab = case
    x, W = V.inputs(tokens, d, vocab, DTYPE[t], 5, dyadic=True)
    x[:, 0] = 1
    W[:, 0] = offset
    return x, W


@pytest.mark.parametrize("name", ROUTES)
def test_loss_does_not_depend_on_an_offset(name):
    """A constant added to every logit changes no loss by a bit (all differences of
    logits are exact), and shifts lse by it to a rounding of lse; every loss is
    within its own roundings of the definition."""
    print("offset", name, flush=True)
    case = ROUTES[name]
    _, tokens, d, vocab = case
    targets = V.draw_targets(tokens, vocab, 6)
    top = 5
    ids, teacher = V.draw_teacher(tokens, vocab, top, 7)
    temperature = 1.5
    got = {}
    for offset in (0.0, 1024.0, -1024.0):
        x, W = _inputs(case, offset)
        got[offset] = (*L.cross_entropy_forward(x, W, targets),
                       *L.distill_forward(x, W, ids, teacher, temperature))
        if offset == 0:
            ref = V.targets_reference(x, W, targets)
            kd = V.teacher_reference(x, W, ids, teacher, temperature)
    loss, lse, kd_loss, kd_lse, z = got[0.0]
    for offset in (1024.0, -1024.0):
        other = got[offset]
        assert torch.equal(other[0], loss) and torch.equal(other[2], kd_loss), offset
        part = targets >= 0
        err = (other[1].double() - ref["lse"] - offset)[part].abs().max().item()
        # L to a few roundings of its own and one addition, below 2^11: half a step
        assert err <= 2.0 ** -14 + 64 * U32 * 16, (offset, err)
    assert bool((loss >= 0).all())
    # (vocab / 128 sums in a thread and 128 roundings in a wave at most, as
    # vocab_cases.lse_tolerance has them; a term's exponent is off by 3 half steps of
    # its distance from the maximum, which the terms weigh: 3 E_p[max - z])
    for value, r, t in ((loss, ref, 1.0), (kd_loss, kd, temperature)):
        p = torch.softmax(r["logits"] / t, 1)
        top_z = r["logits"].max(1).values
        mean = (p * (top_z[:, None] - r["logits"])).sum(1) / t
        tol = U32 * (3 * mean + 128 + vocab / 128)
        if value is loss:
            tol = tol + 4 * U32 * r["loss"]
        else:
            # p to 64 half steps and its sum to `top` more, of terms up to |log p| + (M - z) / T + L
            far = (top_z[:, None] - r["z"]).abs().max(1).values / t + 64
            tol = t * t * (tol + U32 * (64 + top) * far)
        err = (value.double() - r["loss"]).abs()
        print(f"    worst {err.max().item():.2e}, bound there {tol[err.argmax()].item():.2e}",
              flush=True)
        assert bool((err <= tol).all()), (err - tol).max().item()


@pytest.mark.parametrize("name", ROUTES)
def test_one_dominating_logit(name):
    """A row whose other logits are 2000 lower and more: its sum of exponentials is
    exactly 1, lse the logit, and the loss at it exactly 0."""
    print("dominating", name, flush=True)
    t, tokens, d, vocab = ROUTES[name]
    x, W = V.inputs(tokens, d, vocab, DTYPE[t], 8, dyadic=True)
    ids = [0, vocab - 1, vocab // 2, vocab - 200, 300]
    x[:, :len(ids)] = 0
    W[:, :len(ids)] = 0
    row = torch.arange(tokens, device="cuda")
    for k, i in enumerate(ids):
        x[row % len(ids) == k, k] = 1
        W[i, k] = 4096
    target = torch.tensor(ids, device="cuda")[row % len(ids)]
    want = (x.double() * W[target].double()).sum(1)
    assert bool((want == want.float().double()).all())
    loss, lse = L.cross_entropy_forward(x, W, target)
    assert bool((loss == 0).all())
    assert torch.equal(lse.double(), want)
    for temperature in (1.0, 2.0, 1.5):
        teacher = torch.zeros(tokens, 1, device="cuda")
        loss, lse, z = L.distill_forward(x, W, target[:, None].contiguous(), teacher, temperature)
        assert torch.equal(z[:, 0].double(), want)
        assert bool((loss == 0).all()), temperature
        # (1 / T and its product)
        assert bool(((lse.double() - want / temperature).abs() <=
                     2 * U32 * want / temperature).all())


@pytest.mark.parametrize("scale", [1.0, 4.0, 16.0])
@pytest.mark.parametrize("name", ["tiles, float32", "tiles", "rows padded to a tile",
                                  "256 x 256 tiles, last columns on small tiles"])
def test_losses_are_not_negative(name, scale):
    """The target the likeliest id of its row, ordinary values: the loss is never below 0, and
    differs from the exact one of the same logits by roundings of its own size."""
    t, tokens, d, vocab = ROUTES[name]
    x, W = V.inputs(tokens, d, vocab, DTYPE[t], 9)
    x = x * scale
    # (two ways to sum the products may disagree on which is the largest: ask the kernel)
    near = x.float().mm(W.float().t())
    target = near.argmax(1)
    loss, _ = L.cross_entropy_forward(x, W, target)
    # the runner-up within the products' rounding of the largest: by at most that much
    bound = 2 * U32 * (d + 8) * x.double().abs().mm(W.double().abs().t()).max(1).values
    two = near.topk(2, 1).values
    clear = (two[:, 0] - two[:, 1]).double() > 4 * bound
    assert int(clear.sum()) > tokens // 2
    assert bool((loss[clear] >= 0).all()), loss[clear].min().item()


@pytest.mark.parametrize("name", ROUTES)
def test_gradients_do_not_depend_on_an_offset(name):
    """The same constant in every logit and in lse (both exact): the differences that
    the gradients are made of are the same, and so is every bit of g_x and g_W, but
    for the column of W that holds the constant."""
    print("gradients, offset", name, flush=True)
    case = ROUTES[name]
    _, tokens, d, vocab = case
    targets = V.draw_targets(tokens, vocab, 6)
    ids, teacher = V.draw_teacher(tokens, vocab, 5, 7)
    g = (torch.rand(tokens, generator=torch.Generator().manual_seed(3)) + 0.5).cuda()
    x, W = _inputs(case, 0.0)
    # (of the size of the rows' lse, in sixteenths; at T = 2 z / T is exact too)
    _, lse = L.cross_entropy_forward(x, W, targets)
    lse = torch.where(targets >= 0, torch.round(lse * 16) / 16, lse)
    _, kd_lse, _ = L.distill_forward(x, W, ids, teacher, 2.0)
    kd_lse = torch.round(kd_lse * 16) / 16
    got = []
    for offset in (0.0, 1024.0, -1024.0):
        x, W = _inputs(case, offset)
        _, _, z = L.distill_forward(x, W, ids, teacher, 2.0)
        got.append((
            *L.cross_entropy_backward(g, x, W, targets, lse + offset, g_lse=0.25 * g, need_g_W=True),
            *L.distill_backward(g, x, W, ids, teacher, kd_lse + offset / 2, z, 2.0, need_g_W=True)))
    for other in got[1:]:
        for k, (a, b) in enumerate(zip(got[0], other)):
            assert torch.equal(a[:, 1:], b[:, 1:]), (k, (a - b)[:, 1:].abs().max().item())
            assert k % 2 == 0 or torch.equal(a, b)


def test_exponentials_of_float32():
    """g_W of one token whose x is 1 in one column: g_loss exp(z - lse) itself, of logits
    that are exact, from e^-64 to e^64. Within half steps: 2 of the hardware's
    exponential, 1 each of its correction, of the product with g_loss and of the matrix
    product, and 1 of what a correction of second order leaves."""
    vocab = 8193
    z = (torch.arange(vocab, device="cuda") - 4096).double() / 64
    x, W = torch.zeros(1, 8, device="cuda"), torch.zeros(vocab, 8, device="cuda")
    x[0, 0] = 1
    W[:, 0] = z.float()
    target = torch.tensor([0], device="cuda")
    g = torch.full((1,), 0.75, device="cuda")
    for lse in (0.0, 3.0, -5.0):
        _, g_W = L.cross_entropy_backward(g, x, W, target, torch.full((1,), lse, device="cuda"),
                                          need_g_x=False, need_g_W=True)
        want = 0.75 * torch.exp(z - lse)
        err = ((g_W[:, 0].double() - want).abs() / want)[1:]
        print(f"    worst {err.max().item() / U32:.2f} half steps", flush=True)
        assert bool((err <= 6 * U32).all())
    # z / T with an exact 1 / T, and entries of a list among them
    ids = torch.tensor([[5, 4096, 8000]], device="cuda")
    teacher = torch.zeros(1, 3, device="cuda")
    z32 = W[ids[0], 0][None].contiguous()
    _, g_W = L.distill_backward(g, x, W, ids, teacher, torch.full((1,), 2.0, device="cuda"), z32, 4.0,
                                need_g_x=False, need_g_W=True)
    want = 3.0 * torch.exp(z / 4 - 2)
    keep = torch.ones(vocab, dtype=torch.bool, device="cuda")
    keep[ids[0]] = False
    assert bool((((g_W[:, 0].double() - want).abs() / want)[keep] <= 6 * U32).all())


SMALL = 0.75 * 2.0 ** -12  # lost wherever it is added to 4096 (a half step of which is 2^-12)


def test_long_sums_of_float32():
    """One large term and thousands that are below half a step of it: added to it one by
    one they would all be lost. They are summed in blocks of at most 64 before: half a
    step of 4096 for each of the first block's and for each block."""
    def bound(terms):
        return (64 + terms / 64 + 8) * 2.0 ** -12  # (the last blocks are smaller)

    # a logit over d columns, against one that is 4096 exactly
    for tokens in (3, 300):
        d, vocab = 4096, 2
        x = torch.ones(tokens, d, device="cuda")
        W = torch.zeros(vocab, d, device="cuda")
        W[:, 0] = 4096
        W[0, 1:] = SMALL
        more = (d - 1) * SMALL
        targets = torch.zeros(tokens, dtype=torch.int64, device="cuda")
        loss, lse = L.cross_entropy_forward(x, W, targets)
        want = math.log1p(math.exp(-more))
        # (the loss's slope in the logit's difference is below 1)
        assert bool(((loss.double() - want).abs() <= bound(d) + 1e-6).all())
        assert abs(want - math.log(2.0)) > 0.2 > bound(d)
    # g_x over the vocabulary and g_W over the tokens: logits of 0, lse of 0, so that g_z is
    # g_loss but at the targets, whose column of W and row of x are 0
    tokens, d, vocab = 2049, 2048, 8193
    x = torch.zeros(tokens, d, device="cuda")
    W = torch.zeros(vocab, d, device="cuda")
    x[:, :d // 2] = SMALL
    x[0, :d // 2] = 4096
    W[:, d // 2:] = SMALL
    W[0, d // 2:] = 4096
    W[vocab - 1] = 0
    targets = torch.full((tokens,), vocab - 1, device="cuda")
    one, zero = torch.ones(tokens, device="cuda"), torch.zeros(tokens, device="cuda")
    g_x, g_W = L.cross_entropy_backward(one, x, W, targets, zero, need_g_W=True)
    want_x, want_W = 4096 + (vocab - 2) * SMALL, 4096 + (tokens - 1) * SMALL
    assert (vocab - 2) * SMALL > 1.4 and bound(vocab) < 0.2
    assert bool(((g_x[:, d // 2:].double() - want_x).abs() <= bound(vocab)).all())
    assert bool(((g_W[:vocab - 1, :d // 2].double() - want_W).abs() <= bound(tokens)).all())
    assert bool((g_x[:, :d // 2] == 0).all()) and bool((g_W[:, d // 2:] == 0).all())

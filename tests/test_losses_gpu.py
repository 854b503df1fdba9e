"""Softmax cross entropy and distillation without kept logits, against float64
definitions (GPU). Tolerances count roundings; see the functions that form
them."""
import math

import pytest
import torch

from tests import vocab_cases as V

pytestmark = pytest.mark.gpu

L = pytest.importorskip("orthogonal_equivalence_amd.losses",
                        reason="libpoetx.so not built (run the build first)")


def within(name, got, ref, tol):
    """Every element of got within tol (a tensor or number) of ref."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), name
    err = (got.double() - ref).abs()
    over = err - tol
    worst = int(over.argmax())
    print(f"    {name}: worst error {err.max().item():.3e}, nearest the bound: "
          f"{err.flatten()[worst].item():.3e}", flush=True)
    assert bool((over <= 0).all()), (name, worst, err.flatten()[worst].item())


def forward_tolerances(ref, temperature, d, x, W, dyadic, p=None):
    """lse and loss: the loss adds T^2 (weights that sum to 1) times lse's error,
    z's own, and a few half steps of its terms."""
    u = 2.0 ** -24
    lse = V.lse_tolerance(ref, temperature, d, x, W, dyadic)
    z = torch.zeros_like(lse) if dyadic else \
        2 * u * (d + 8) * x.double().abs().mm(W.double().abs().t()).max(1).values
    big = ref["logits"].abs().max(1).values / temperature + ref["lse"].abs() + 64
    loss = temperature ** 2 * (lse + z / temperature + 16 * u * big)
    return lse, z, loss


def gradient_tolerances(ref, x, W, dtype, temperature, part, listed):
    """g_z to a half step of its type (the products' operand) and what float32
    loses before: the exponent's roundings and the listed entries' p (`listed`: terms in
    a sum of p, each off by a few half steps). Then the products: one step of
    float32 a term, and the result's rounding."""
    u, h = 2.0 ** -24, V.HALF[dtype]
    rows = ref["logits"].abs().max(1).values / temperature + ref["lse"].abs() + 16 + 4 * listed
    # (p and the target's part cancel in g_z: both count)
    mag = ref["mag"]
    e_z = ref["g_z"].abs() * h + mag * (u * 4) * rows[:, None] + \
        mag * (0.0 if ref["dyadic"] else 2 * u * (x.shape[1] + 8)) * ref["bound"][:, None]
    xs = torch.where(part[:, None], x.double(), torch.zeros_like(x.double())).abs()
    Wa = W.double().abs()
    tol_x = e_z.mm(Wa) + 2 * u * (W.shape[0] + 16) * ref["g_z"].abs().mm(Wa) + \
        2 * h * ref["g_x"].abs()
    tol_W = e_z.t().mm(xs) + 2 * u * (x.shape[0] + 16) * ref["g_z"].abs().t().mm(xs) + \
        2 * h * ref["g_W"].abs()
    return tol_x + 1e-30, tol_W + 1e-30


def magnitudes(ref, g_loss, a, temperature, part, ids, p, lse, dyadic, x, W):
    """|a| exp(z / T - lse) + the listed parts: what g_z is the difference of."""
    z = ref["logits"]
    m = torch.exp(z / temperature - lse.double()[:, None]) * a.double().abs()[:, None]
    m = torch.where(part[:, None], m, torch.zeros_like(m))
    m.scatter_add_(1, ids.clamp(min=0), torch.where(
        ids >= 0, (g_loss.double().abs() * temperature)[:, None] * p, torch.zeros_like(p)))
    ref["mag"], ref["dyadic"] = m, dyadic
    ref["bound"] = x.double().abs().mm(W.double().abs().t()).max(1).values / temperature
    return ref


SIZES = [  # tokens, d, vocab
    (1, 8, 1), (1, 64, 7), (1, 2048, 5000), (2, 72, 33), (3, 256, 256), (16, 128, 1000),
    (17, 200, 257), (64, 256, 1000), (100, 264, 513), (255, 64, 2049), (256, 256, 512),
    (300, 512, 4099), (777, 96, 1031), (20, 136, 30011), (40, 256, 20000), (64, 1032, 9000),
    (7, 40, 100003),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dyadic", [True, False])
@pytest.mark.parametrize("tokens,d,vocab", SIZES)
def test_cross_entropy(tokens, d, vocab, dyadic, dtype):
    print(f"cross entropy {tokens} {d} {vocab} {dtype} dyadic={dyadic}", flush=True)
    x, W = V.inputs(tokens, d, vocab, dtype, 1, dyadic)
    t = V.draw_targets(tokens, vocab, 2)
    loss, lse = L.cross_entropy_forward(x, W, t)
    ref = V.targets_reference(x, W, t)
    tol_lse, _, tol_loss = forward_tolerances(ref, 1.0, d, x, W, dyadic)
    within("lse", lse, ref["lse"], tol_lse)
    within("loss", loss, ref["loss"], tol_loss)
    assert bool((loss[t < 0] == 0).all()) and bool((lse[t < 0] == 0).all())

    gen = torch.Generator().manual_seed(3)
    g = (torch.rand(tokens, generator=gen) + 0.5).cuda()
    for g_lse in (None, torch.randn(tokens, generator=gen).cuda()):
        ref = V.targets_reference(x, W, t, g_loss=g, g_lse=g_lse, lse=lse)
        part = t >= 0
        a = g if g_lse is None else g + g_lse
        magnitudes(ref, g, a, 1.0, part, t[:, None], part.double()[:, None], lse, dyadic, x, W)
        tol_x, tol_W = gradient_tolerances(ref, x, W, dtype, 1.0, part, 1)
        g_x, g_W = L.cross_entropy_backward(g, x, W, t, lse, g_lse=g_lse, need_g_W=True)
        within("g_x", g_x, ref["g_x"], tol_x)
        within("g_W", g_W, ref["g_W"], tol_W)
        assert bool((g_x[t < 0] == 0).all())
        # (alone, a product may be cut into other partial sums than beside the other)
        only, none = L.cross_entropy_backward(g, x, W, t, lse, g_lse=g_lse)
        assert none is None
        within("g_x alone", only, ref["g_x"], tol_x)
        none, only = L.cross_entropy_backward(g, x, W, t, lse, g_lse=g_lse, need_g_x=False,
                                              need_g_W=True)
        assert none is None
        within("g_W alone", only, ref["g_W"], tol_W)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,d,vocab,top,temperature,dyadic", [
    # (the longer lists get their logits out of the products)
    (1126, 2832, 501, 59, 1.0, True), (1000, 1024, 8333, 128, 2.0, True),
    (600, 512, 20000, 400, 1.0, False), (300, 1024, 2000, 600, 1.5, True),
    (1, 8, 1, 1, 1.0, True), (1, 64, 50, 3, 2.0, True), (5, 72, 33, 40, 0.5, True),
    (16, 128, 1000, 8, 1.0, True), (33, 256, 257, 64, 4.0, False), (100, 264, 2049, 65, 1.5, True),
    (300, 512, 4099, 5, 2.0, False), (40, 64, 3000, 1024, 1.0, True), (256, 256, 512, 17, 1.0, True),
])
def test_distill(tokens, d, vocab, top, temperature, dyadic, kind, dtype):
    print(f"distill {tokens} {d} {vocab} {top} {temperature} {kind} {dtype}", flush=True)
    x, W = V.inputs(tokens, d, vocab, dtype, 1, dyadic)
    ids, teacher = V.draw_teacher(tokens, vocab, top, 2, kind)
    loss, lse, z = L.distill_forward(x, W, ids, teacher, temperature)
    ref = V.teacher_reference(x, W, ids, teacher, temperature)
    tol_lse, tol_z, tol_loss = forward_tolerances(ref, temperature, d, x, W, dyadic)
    within("lse", lse, ref["lse"], tol_lse)
    within("z", z, ref["z"], tol_z[:, None] + 0 * ref["z"])
    # (p: its logits' differences, up to ~30, rounded once, and sums of `top` terms)
    within("loss", loss, ref["loss"], tol_loss * 2 + temperature ** 2 * 2.0 ** -24 * (
        64 + top) * (ref["loss"].abs() / temperature ** 2 + 64))

    g = (torch.rand(tokens, generator=torch.Generator().manual_seed(3)) + 0.5).cuda()
    ref = V.teacher_reference(x, W, ids, teacher, temperature, g_loss=g, lse=lse)
    held = (ids >= 0) & (teacher > -math.inf)
    part = held.any(1)
    t64 = torch.where(held, teacher.double() / temperature, torch.tensor(-math.inf).double().cuda())
    p = torch.where(part[:, None], torch.softmax(t64, 1), torch.zeros_like(t64)).nan_to_num(0.0)
    magnitudes(ref, g, g * temperature, temperature, part, ids, p, lse, dyadic, x, W)
    tol_x, tol_W = gradient_tolerances(ref, x, W, dtype, temperature, part, min(top, 32) + 64)
    g_x, g_W = L.distill_backward(g, x, W, ids, teacher, lse, z, temperature, need_g_W=True)
    within("g_x", g_x, ref["g_x"], tol_x)
    within("g_W", g_W, ref["g_W"], tol_W)
    assert bool((g_x[~part] == 0).all()) and bool((loss[~part] == 0).all())
    only, none = L.distill_backward(g, x, W, ids, teacher, lse, z, temperature)
    assert none is None
    within("g_x alone", only, ref["g_x"], tol_x)


def counted(tokens, d, vocab, seed, dtype=torch.bfloat16):
    """Operands whose logits are all 0 (x lives in the first half of the
    columns, W in the second) and whose gradients are integers: with
    g_loss = b and g_lse = vocab - b the logits' gradient is 1, and 1 - b at
    the target (vocab exp(-lse) is within 2^-20 of 1, which bf16 rounds to 1)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = d // 2
    x = torch.zeros(tokens, d, device="cuda", dtype=dtype)
    W = torch.zeros(vocab, d, device="cuda", dtype=dtype)
    x[:, :h] = torch.randint(-2, 3, (tokens, h), generator=gen, device="cuda").to(dtype)
    W[:, h:] = torch.randint(-1, 2, (vocab, d - h), generator=gen, device="cuda").to(dtype)
    t = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    t[torch.rand(tokens, generator=gen, device="cuda") < 0.2] = -100
    t[0] = vocab - 1
    return x, W, t


@pytest.mark.parametrize("tokens,d,vocab", [
    (1, 64, 4096), (31, 128, 30000), (300, 256, 5003), (512, 512, 2048), (777, 256, 50001),
    (1000, 320, 20483), (2048, 64, 131072), (2304, 256, 131072), (4100, 96, 65537),
    (9000, 64, 131072), (515, 1064, 3001), (64, 512, 40001), (5, 4096, 9001), (40, 72, 131072),
    (33, 2056, 20001),
    # (g_x whole in one product, with and without a ragged last K tile; columns
    # shifted back; several pieces with them)
    (8192, 2048, 515), (8192, 2048, 1024), (777, 352, 20003), (2304, 288, 131072),
    (300, 4096, 3001), (256, 256, 256), (257, 2080, 777),
])
def test_counted_operands(tokens, d, vocab):
    """Every element of loss, lse, g_x and g_W of large and ragged sizes (several
    pieces of the vocabulary, several ranges of rows) on integer operands: a
    lost, doubled or shifted row, column or piece shows at once."""
    print(f"counted {tokens} {d} {vocab}", flush=True)
    x, W, t = counted(tokens, d, vocab, 7)
    part = t >= 0
    loss, lse = L.cross_entropy_forward(x, W, t)
    # the sum of exponentials is the integer vocab, exact; its logarithm, the product and
    # the stored value round once each
    want = torch.where(part, math.log(vocab), 0.0).double()
    assert bool(((lse.double() - want).abs() <= 4 * 2.0 ** -24 * math.log(vocab)).all())
    assert torch.equal(loss, lse)  # less a logit of 0
    b = 3.0
    g_loss = torch.full((tokens,), b, device="cuda")
    g_lse = torch.full((tokens,), vocab - b, device="cuda")
    g_x, g_W = L.cross_entropy_backward(g_loss, x, W, t, lse, g_lse=g_lse, need_g_W=True)
    # integers: sums in float64, rounded once to bf16
    Wd, xd = W.double(), torch.where(part[:, None], x.double(), 0.0)
    want_x = torch.where(part[:, None], Wd.sum(0) - b * Wd[t.clamp(min=0)], 0.0)
    assert torch.equal(g_x.double(), want_x.float().bfloat16().double())
    want_W = xd.sum(0).expand(vocab, d).clone()
    want_W.index_add_(0, t.clamp(min=0), -b * xd)
    assert torch.equal(g_W.double(), want_W.float().bfloat16().double())


@pytest.mark.parametrize("case", V.CASES, ids=str)
def test_every_variant(case):
    """Both directions on operands whose results are whole numbers, every element:
    as above, with an lse of 0 given to the backward, so that exp(z - lse) is 1
    to the last bit in both types."""
    print("variant", case, flush=True)
    t, tokens, d, vocab = case
    dtype = torch.bfloat16 if t == V.BF16 else torch.float32
    x, W, target = counted(tokens, d, vocab, 11, dtype)
    part = target >= 0
    loss, lse = L.cross_entropy_forward(x, W, target)
    want = torch.where(part, math.log(vocab), 0.0).double()
    assert bool(((lse.double() - want).abs() <= 4 * 2.0 ** -24 * math.log(vocab)).all())
    assert torch.equal(loss, lse)
    g_loss = torch.full((tokens,), 3.0, device="cuda")
    g_x, g_W = L.cross_entropy_backward(g_loss, x, W, target, torch.zeros_like(lse),
                                        g_lse=g_loss * 0 - 2.0, need_g_W=True)
    Wd, xd = W.double(), torch.where(part[:, None], x.double(), 0.0)
    want_x = torch.where(part[:, None], Wd.sum(0) - 3 * Wd[target.clamp(min=0)], 0.0)
    assert torch.equal(g_x, want_x.float().to(dtype))
    want_W = xd.sum(0).expand(vocab, d).clone()
    want_W.index_add_(0, target.clamp(min=0), -3 * xd)
    assert torch.equal(g_W, want_W.float().to(dtype))


@pytest.mark.parametrize("case", V.LISTED, ids=str)
def test_every_listed_variant(case):
    t, tokens, d, vocab, top = case
    test_distill(tokens, d, vocab, top, 1.0, True, "f32", "bf16" if t == V.BF16 else "f32")


def test_rows_that_take_no_part():
    """Padding may hold anything: NaN and infinities in the x of an ignored row
    reach no other row's results and no gradient; a batch of nothing but such
    rows gives zeros."""
    for dtype in ("f32", "bf16"):
        x, W = V.inputs(300, 256, 1000, dtype, 1, True)
        t = V.draw_targets(300, 1000, 2, ignored=0.5)
        clean = torch.where((t >= 0)[:, None], x, torch.zeros_like(x))
        dirty = clean.clone()
        dirty[t < 0] = torch.tensor([math.nan, math.inf, -math.inf, 3e38] * 64).to(dirty.dtype).cuda()
        a, b = (L.cross_entropy_forward(v, W, t) for v in (clean, dirty))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        g = torch.ones(300, device="cuda")
        a, b = (L.cross_entropy_backward(g, v, W, t, a[1], need_g_W=True) for v in (clean, dirty))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        none = torch.full_like(t, -100)
        loss, lse = L.cross_entropy_forward(dirty, W, none)
        g_x, g_W = L.cross_entropy_backward(g, dirty, W, none, lse, g_lse=g, need_g_W=True)
        for v in (loss, lse, g_x, g_W):
            assert bool((v == 0).all())
        ids = torch.where((t >= 0)[:, None], t[:, None], -1).expand(300, 3).contiguous()
        teacher = torch.zeros(300, 3, device="cuda")
        out = []
        for v in (clean, dirty):
            loss, lse, z = L.distill_forward(v, W, ids, teacher, 2.0)
            out.append((loss, lse, z, *L.distill_backward(g, v, W, ids, teacher, lse, z, 2.0,
                                                          need_g_W=True)))
        assert all(torch.equal(p, q) for p, q in zip(*out))


def test_teacher_masks():
    """Entries masked by -inf, by the type's lowest value and by a negative id
    are the same distribution; a row of lowest values alone is uniform."""
    x, W = V.inputs(64, 128, 999, "bf16", 1, True)
    gen = torch.Generator().manual_seed(5)
    ids = torch.randint(0, 999, (64, 6), generator=gen).cuda()
    t = torch.randn(64, 6, generator=gen).cuda()
    ref = None
    for how in ("id", "inf", "low"):
        i, v = ids.clone(), t.clone()
        if how == "id":
            i[:, 4:] = -1
        else:
            v[:, 4:] = -math.inf if how == "inf" else torch.finfo(torch.float32).min
        loss, lse, z = L.distill_forward(x, W, i, v, 0.5)
        g = torch.ones(64, device="cuda")
        got = (loss, lse, *L.distill_backward(g, x, W, i, v, lse, z, 0.5, need_g_W=True))
        if ref is None:
            ref = got
        assert all(torch.equal(p, q) for p, q in zip(ref, got)), how
    low = torch.full_like(t, torch.finfo(torch.float32).min)
    a = L.distill_forward(x, W, ids, low)
    b = L.distill_forward(x, W, ids, torch.zeros_like(t))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_ids_past_the_vocabulary():
    """Read nowhere; the row's loss is NaN and so are the gradients."""
    x, W = V.inputs(40, 64, 100, "bf16", 1, True)
    t = V.draw_targets(40, 100, 2, ignored=0)
    for bad in (100, 101, 2 ** 31, 2 ** 40, 2 ** 62):
        t2 = t.clone()
        t2[7] = bad
        loss, lse = L.cross_entropy_forward(x, W, t2)
        assert bool(torch.isnan(loss[7])) and int(torch.isnan(loss).sum()) == 1
        g_x, g_W = L.cross_entropy_backward(torch.ones(40, device="cuda"), x, W, t2, lse,
                                            need_g_W=True)
        assert bool(torch.isnan(g_x[7]).all()) and int(torch.isnan(g_x).sum()) == 64
        assert bool(torch.isnan(g_W).any())
        ids = t2[:, None].expand(40, 2).contiguous()
        loss, lse, z = L.distill_forward(x, W, ids, torch.zeros(40, 2, device="cuda"))
        assert bool(torch.isnan(loss[7])) and int(torch.isnan(loss).sum()) == 1
        g_x, _ = L.distill_backward(torch.ones(40, device="cuda"), x, W, ids,
                                    torch.zeros(40, 2, device="cuda"), lse, z)
        assert bool(torch.isnan(g_x[7]).all()) and int(torch.isnan(g_x).sum()) == 64


@pytest.mark.parametrize("tokens,d,vocab,top", [(700, 512, 9000, 512), (130, 4096, 700, 300)])
def test_lists_in_one_place(tokens, d, vocab, top):
    """Every id of every row within a few columns (one wave's cell holds thousands
    of entries), one of them past the vocabulary: each entry's own logit, exact."""
    x, W = V.inputs(tokens, d, vocab, "bf16", 1, True)
    gen = torch.Generator().manual_seed(9)
    ids = torch.randint(0, 5, (tokens, top), generator=gen).cuda()
    ids[:, 7] = vocab - 1
    ids[3, 5] = vocab
    ids[4, 6] = -7
    teacher = torch.randn(tokens, top, generator=gen).cuda()
    loss, lse, z = L.distill_forward(x, W, ids, teacher)
    want = x.double().mm(W.double().t()).gather(1, ids.clamp(0, vocab - 1))
    want[4, 6] = 0
    assert bool(torch.isnan(z[3, 5])) and bool(torch.isnan(loss[3]))
    want[3, 5] = z[3, 5] = 0
    assert torch.equal(z.double(), want)
    assert int(torch.isnan(loss).sum()) == 1


def test_large_and_infinite_logits():
    """Logits of +-1e4 and beyond neither overflow nor lose the sum; infinities
    and NaN stay in their own rows."""
    x, W = V.inputs(33, 64, 700, "f32", 1, True)
    x = x * 4096
    t = V.draw_targets(33, 700, 2, ignored=0)
    loss, lse = L.cross_entropy_forward(x, W, t)
    ref = V.targets_reference(x, W, t)
    tol, _, tol_loss = forward_tolerances(ref, 1.0, 64, x, W, True)
    within("lse", lse, ref["lse"], tol)
    within("loss", loss, ref["loss"], tol_loss)
    bad = x.clone()
    bad[5, 3] = math.nan
    bad[6, 4] = math.inf
    loss2, lse2 = L.cross_entropy_forward(bad, W, t)
    keep = [i for i in range(33) if i not in (5, 6)]
    assert torch.equal(loss2[keep], loss[keep]) and torch.equal(lse2[keep], lse[keep])
    assert bool(torch.isnan(loss2[5])) and not bool(torch.isfinite(loss2[6]))
    # a logit of +inf: lse is +inf; of -inf: its term is 0
    W2 = torch.zeros(700, 64, device="cuda")
    x2 = torch.ones(2, 64, device="cuda")
    W2[9, 0] = math.inf
    W2[10, 0] = -math.inf
    x2[1, 0] = 0
    x3 = x2[:1]
    W2[9, 0] = -math.inf
    loss3, lse3 = L.cross_entropy_forward(x3, W2, torch.tensor([3], device="cuda"))
    assert abs(lse3.item() - math.log(698)) <= 4 * 2.0 ** -24 * math.log(698)
    W2[9, 0] = math.inf
    _, lse3 = L.cross_entropy_forward(x3, W2, torch.tensor([3], device="cuda"))
    assert lse3.item() == math.inf


@pytest.mark.parametrize("dtype", ["f32"])
def test_gradients_against_differences(dtype):
    """g_x and g_W against central differences of the float64 loss at the same
    operands (step 2^-10 of values of order 1: the differences are off by the
    third derivative times 2^-20 / 6, the derivatives of order 1)."""
    tokens, d, vocab, T = 6, 16, 40, 2.0
    x, W = V.inputs(tokens, d, vocab, dtype, 1)
    ids, teacher = V.draw_teacher(tokens, vocab, 5, 4)
    t = V.draw_targets(tokens, vocab, 2)
    g = (torch.rand(tokens, generator=torch.Generator().manual_seed(3)) + 0.5).cuda()
    cases = []
    _, lse = L.cross_entropy_forward(x, W, t)
    g_lse = 0.1 * g
    cases.append((L.cross_entropy_backward(g, x, W, t, lse, g_lse=g_lse, need_g_W=True),
                  lambda a, b: (lambda r: (r["loss"] * g.double()).sum() +
                                (r["lse"] * g_lse.double()).sum())(V.targets_reference(a, b, t))))
    _, lse2, z = L.distill_forward(x, W, ids, teacher, T)
    cases.append((L.distill_backward(g, x, W, ids, teacher, lse2, z, T, need_g_W=True),
                  lambda a, b: (V.teacher_reference(a, b, ids, teacher, T)["loss"] *
                                g.double()).sum()))
    h = 2.0 ** -10
    for (g_x, g_W), f in cases:
        for which, grad in ((0, g_x), (1, g_W)):
            base = [x.double(), W.double()]
            for i, j in ((0, 0), (1, 3), (tokens - 1, d - 1), (3, 7)):
                if which == 1:
                    i = int(ids[0, 0]) if i == 0 else i
                lo, hi = [b.clone() for b in base], [b.clone() for b in base]
                lo[which][i, j] -= h
                hi[which][i, j] += h
                diff = ((f(*hi) - f(*lo)) / (2 * h)).item()
                assert abs(diff - grad[i, j].item()) <= 2e-5, (which, i, j, diff, grad[i, j].item())

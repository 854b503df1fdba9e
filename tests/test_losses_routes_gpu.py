"""Every route of the losses over a vocabulary (vocab_routes.py) on logits that are
not zero: against the float64 definitions, from workspaces that hold NaN, in
ranges of rows, and bit for bit again in repeated calls, on two streams at once
and in graphs (GPU)."""
import math

import pytest
import torch

from tests import test_losses_gpu as G
from tests import vocab_cases as V
from tests.vocab_routes import DTYPE, RANGES, ROUTES, SORTED

pytestmark = pytest.mark.gpu

L = pytest.importorskip("orthogonal_equivalence_amd.losses",
                        reason="libpoetx.so not built (run the build first)")
from orthogonal_equivalence_amd import poetx as P  # noqa: E402

T = 2.0
ALL = {**{n: (*c, 20) for n, c in ROUTES.items()}, **SORTED}


@pytest.mark.parametrize("name", ROUTES)
def test_cross_entropy(name):
    t, tokens, d, vocab = ROUTES[name]
    G.test_cross_entropy(tokens, d, vocab, True, DTYPE[t])


@pytest.mark.parametrize("name", ALL)
def test_distill(name):
    t, tokens, d, vocab, top = ALL[name]
    G.test_distill(tokens, d, vocab, top, T, True, "f32", DTYPE[t])


def _args(name, seed):
    t, tokens, d, vocab, top = ALL[name]
    x, W = V.inputs(tokens, d, vocab, DTYPE[t], seed)
    g = (torch.rand(tokens, generator=torch.Generator().manual_seed(seed)) + 0.5).cuda()
    return (g, x, W, V.draw_targets(tokens, vocab, seed + 10),
            *V.draw_teacher(tokens, vocab, top, seed + 20))


def _all(g, x, W, targets, ids, teacher, stream=None):
    """Every output of the four calls, with and without g_W and a gradient to lse."""
    loss, lse = L.cross_entropy_forward(x, W, targets, stream=stream)
    out = [loss, lse, *L.cross_entropy_backward(g, x, W, targets, lse, need_g_W=True, stream=stream)]
    out += L.cross_entropy_backward(g, x, W, targets, lse, g_lse=g, stream=stream)[:1]
    loss, lse, z = L.distill_forward(x, W, ids, teacher, T, stream=stream)
    out += [loss, lse, z]
    out += L.distill_backward(g, x, W, ids, teacher, lse, z, T, need_g_W=True, stream=stream)
    return out + [L.distill_backward(g, x, W, ids, teacher, lse, z, T, stream=stream)[0]]


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("name", ALL)
def test_repeated(name):
    print("repeated", name, flush=True)
    args = _args(name, 1)
    ref = _all(*args)
    assert all(bool(torch.isfinite(v).all()) for v in ref)
    for k in range(3):
        # (other data in the memory that the next calls are given)
        junk = [torch.full_like(v, math.nan) for v in ref]
        del junk
        assert _same(ref, _all(*args)), k


@pytest.mark.parametrize("name", ALL)
def test_two_streams_at_once(name):
    print("streams", name, flush=True)
    sides = []
    for seed in (1, 2):
        args = _args(name, seed)
        sides.append((args, _all(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[_all(*args, stream=s) for args, _, s in sides] for _ in range(2)]
    torch.cuda.synchronize()
    for row in got:
        for (_, ref, _), out in zip(sides, row):
            assert _same(ref, out)


@pytest.mark.parametrize("name", ALL)
def test_graphs(name):
    """Two graphs of the four calls, replayed in turn on new inputs between eager calls."""
    print("graphs", name, flush=True)
    first, second = _args(name, 1), _args(name, 2)
    _all(*first)
    torch.cuda.synchronize()
    sides = []
    for _ in range(2):
        own = [v.clone() for v in first]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = _all(*own)
        sides.append((own, graph, got))
    for k in range(4):
        own, graph, got = sides[k % 2]
        for a, b in zip(own, second if k in (0, 3) else first):
            a.copy_(b)
        graph.replay()
        ref = _all(*[v.clone() for v in own])
        torch.cuda.synchronize()
        assert _same(got, ref), k


def _guarded(nbytes):
    """A workspace of NaN of exactly that size, and the bytes behind it."""
    whole = torch.full((nbytes + 4096,), 0xff, dtype=torch.uint8, device="cuda")
    return whole[:nbytes], whole[nbytes:]


@pytest.mark.parametrize("name", ALL)
def test_workspace_of_nan(name):
    """Workspaces of exactly the size that is asked for, and outputs, that hold NaN
    before the call: the same bits, and nothing is written behind them."""
    print("workspace", name, flush=True)
    t, tokens, d, vocab, top = ALL[name]
    args = g, x, W, targets, ids, teacher = _args(name, 3)
    ref = _all(*args)
    act = P.POETX_BF16 if t == V.BF16 else P.POETX_F32
    ends = []

    def out(like):
        whole = torch.full((like.numel() + 64,), math.nan, dtype=like.dtype, device="cuda")
        ends.append(whole[like.numel():])
        return whole[:like.numel()].view(like.shape)

    def space(size, desc):
        ws, end = _guarded(size(desc))
        ends.append(end)
        return ws

    ce = P.make_vocab_desc(tokens, d, vocab, act)
    kd = P.make_vocab_desc(tokens, d, vocab, act, top, P.POETX_F32, T)
    fwd, bwd = P.poetx_vocab_fwd_workspace_size, P.poetx_vocab_bwd_workspace_size
    got = [out(v) for v in ref]
    P.poetx_cross_entropy_fwd(ce, x, W, targets, got[0], got[1], space(fwd, ce))
    P.poetx_cross_entropy_bwd(ce, g, None, x, W, targets, got[1], got[2], got[3], space(bwd, ce))
    P.poetx_cross_entropy_bwd(ce, g, g, x, W, targets, got[1], got[4], None, space(bwd, ce))
    P.poetx_distill_fwd(kd, x, W, ids, teacher, got[5], got[6], got[7], space(fwd, kd))
    P.poetx_distill_bwd(kd, g, x, W, ids, teacher, got[6], got[7], got[8], got[9], space(bwd, kd))
    P.poetx_distill_bwd(kd, g, x, W, ids, teacher, got[6], got[7], got[10], None, space(bwd, kd))
    torch.cuda.synchronize()
    assert _same(ref, got)
    for end in ends:
        assert bool((end == 0xff).all() if end.dtype == torch.uint8 else torch.isnan(end).all())


@pytest.mark.parametrize("name", RANGES)
def test_rows_in_ranges(name):
    """The forward a range of rows at a time, against the definition in float64 by pieces
    of the vocabulary: logits in eighths, exact in float32, at every listed id; every
    loss within its own roundings."""
    print("ranges", name, flush=True)
    _, tokens, d, vocab, top = RANGES[name]
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(-1, 2, (tokens, d), generator=gen, device="cuda").bfloat16()
    W = torch.randint(-3, 4, (vocab, d), generator=gen, device="cuda", dtype=torch.int8).bfloat16() / 8
    ids = torch.randint(0, vocab, (tokens, max(top, 1)), generator=gen, device="cuda")
    ids[:, 0] = torch.where(torch.rand(tokens, generator=gen, device="cuda") < 0.1, -1, ids[:, 0])
    ids[tokens - 1, 0], ids[tokens - 97, 0], ids[tokens - 255, 0] = vocab - 1, 0, vocab // 2
    lse64 = torch.full((tokens,), -math.inf, device="cuda", dtype=torch.float64)
    largest = lse64.clone()
    temperature = T if top else 1.0
    for a in range(0, vocab, 65536):
        z = x.float().mm(W[a:a + 65536].float().t()).double()
        largest = torch.maximum(largest, z.max(1).values)
        lse64 = torch.logaddexp(lse64, torch.logsumexp(z / temperature, 1))
    want = torch.empty(ids.shape, device="cuda")
    for a in range(0, tokens, 100):
        want[a:a + 100] = (W[ids[a:a + 100].clamp(min=0)].float() * x[a:a + 100, None].float()).sum(2)
    want[ids < 0] = 0
    if top:
        teacher = torch.randn(tokens, top, generator=gen, device="cuda")
        loss, lse, z = L.distill_forward(x, W, ids, teacher, T)
        assert torch.equal(z, want)
        held = ids >= 0
        log_p = torch.where(held, teacher.double() / T, -math.inf).log_softmax(1)
        p = log_p.exp()
        log_p = torch.where(held, log_p, 0.0)
        ref = T * T * (p * (log_p - want.double() / T + lse64[:, None])).sum(1)
        part = held.any(1)
    else:
        loss, lse = L.cross_entropy_forward(x, W, ids[:, 0].contiguous())
        part = ids[:, 0] >= 0
        ref = lse64 - want[:, 0].double()
    ref, lse64 = torch.where(part, ref, 0.0), torch.where(part, lse64, 0.0)
    # as in test_losses_rounding_gpu.py: 3 half steps of a term's distance from the maximum,
    # 128 roundings in a wave, 2 in a row's join for each of its vocab / 128 sums over 256 threads,
    # then of the result (and p: 64 + top, of terms up to |log p| + (M - z) / T + L)
    u = 2.0 ** -24
    far = (largest[:, None] - want.double()).abs().max(1).values + 64
    tol = u * (3 * far + 128 + vocab / 128 / 64 + 4 * ref.abs())
    if top:
        tol = T * T * (tol + u * (64 + top) * far)
    err = (loss.double() - ref).abs()
    print(f"    worst {err.max().item():.2e}, bound {tol[err.argmax()].item():.2e}", flush=True)
    assert bool((err <= tol).all())
    assert bool(((lse.double() - lse64).abs() <= tol + 2 * u * lse64).all())

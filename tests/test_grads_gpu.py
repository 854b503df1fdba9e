"""grad_norm and clip_grads against float64 sums. Tolerances: the norm is a
float64 sum rounded once to float32 (2^-24 relative; 2^-23 asserted, for the
float64 steps' own 1e-13), the factor max_norm / norm another such rounding,
the product a third: 3 * 2^-24 relative in float32, and in bfloat16 half a
step, 2^-8, of the value."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here is gpu-marked
    pytest.skip("no GPU", allow_module_level=True)

from orthogonal_equivalence_amd import poetx as P  # noqa: E402
from orthogonal_equivalence_amd.grads import clip_grads, grad_norm  # noqa: E402

F, B = torch.float32, torch.bfloat16


def make(sizes, seed=0, scale=1.0, offset=0):
    """Separate tensors (offset: elements into their allocation)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, (n, dt) in enumerate(sizes):
        t = torch.randn(n + offset, generator=g, device="cuda") * (scale * (1 + i % 3))
        out.append(t.to(dt)[offset:])
    return out


def norm64(grads):
    return math.sqrt(sum(g.double().square().sum().item() for g in grads))


def check_clip(grads, max_norm, outs=None):
    ref = [g.clone() for g in grads]
    n64 = norm64(ref)
    norm = clip_grads(grads, max_norm, outs=outs)
    got = grads if outs is None else outs
    assert norm.shape == () and norm.dtype == F
    assert abs(norm.item() - n64) <= 2.0 ** -23 * n64
    k = max_norm / n64 if n64 > max_norm else 1.0
    for a, r in zip(got, ref):
        want = r.double() * k
        half = 3 * 2.0 ** -24 if r.dtype == F else 2.0 ** -8 + 2.0 ** -22
        # (2^-149: the last step of float32 and, below 2^-126, of bfloat16's 2^-133)
        tiny = 2.0 ** -149 if r.dtype == F else 2.0 ** -133
        if k == 1.0:
            assert torch.equal(a, r)
        else:
            assert ((a.double() - want).abs() <= half * want.abs() + tiny).all()
    if outs is not None:
        assert all(torch.equal(g, r) for g, r in zip(grads, ref))
    return norm


LISTS = {
    "one": [(1, F)], "one_bf16": [(1, B)], "three": [(3, F), (1, B), (5, F)],
    "vectors": [(4096, F), (8192, B), (4095, F), (4097, F), (8191, B), (8193, B)],
    "generators": [(8 * 32640, F), (16 * 32640, F), (2048, F), (2048, B)],
    "odd": [(100003, F), (77777, B), (1, F), (33, B), (500009, F)],
    "empty_among": [(0, F), (10, F), (0, B), (7, B), (0, F)],
    "many": [(257 + 13 * (i % 7), F if i % 3 else B) for i in range(300)],
    "large": [(20_000_003, F), (9_000_001, B)],
}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("offset", [0, 1])
def test_clip(name, offset):
    sizes = LISTS[name]
    print(f"  {name} offset={offset}", flush=True)
    n64 = norm64(make(sizes, offset=offset))
    check_clip(make(sizes, offset=offset), 0.37 * n64)           # in place
    check_clip(make(sizes, offset=offset), 2.0 * n64)            # nothing to clip
    g = make(sizes, offset=offset)
    check_clip(g, 0.37 * n64, outs=[torch.full_like(t, 9.0) for t in g])
    check_clip(g, 2.0 * n64, outs=[torch.full_like(t, 9.0) for t in g])
    check_clip(g, math.inf)
    assert abs(grad_norm(g).item() - n64) <= 2.0 ** -23 * n64
    assert torch.equal(grad_norm(g), grad_norm(g))


def test_views_of_flat_buffers():
    """Neighbouring views, views with gaps (whose values stay) and a list out
    of memory order."""
    flat = torch.randn(70_001, device="cuda")
    keep = flat.clone()
    views = [flat[0:10_000], flat[10_000:10_001], flat[10_001:30_003], flat[40_000:40_007],
             flat[60_000:70_001], flat[50_000:50_500]]
    n = norm64(views)
    check_clip(views, 0.5 * n)
    gaps = [slice(30_003, 40_000), slice(40_007, 50_000), slice(50_500, 60_000)]
    assert all(torch.equal(flat[s], keep[s]) for s in gaps)
    out = torch.full((70_001,), 3.0, device="cuda", dtype=B)
    half = keep.to(B)
    sl = [slice(0, 5), slice(5, 4_000), slice(4_001, 70_000)]
    check_clip([half[s] for s in sl], 10.0, outs=[out[s] for s in sl])
    assert out[4_000] == 3.0 and out[70_000] == 3.0


def test_no_tensors_and_zero_gradients():
    assert clip_grads([], 1.0).item() == 0.0 and grad_norm([]).item() == 0.0
    z = [torch.zeros(5000, device="cuda"), torch.zeros(0, device="cuda")]
    assert clip_grads(z, 1.0).item() == 0.0 and not z[0].any()
    assert clip_grads(z, 0.0).item() == 0.0
    g = [torch.ones(100, device="cuda")]
    assert clip_grads(g, 0.0).item() == 10.0 and not g[0].any()


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e25, 1e36])
def test_values_whose_squares_leave_float32(scale):
    g = make([(1000, F), (333, B), (5001, F)], seed=3, scale=scale)
    check_clip(g, 0.25 * norm64(g))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_not_finite_leaves_the_values(bad):
    g = make([(5000, F), (333, B)], seed=4)
    g[0][4999] = bad
    ref = [t.clone() for t in g]
    norm = clip_grads(g, 0.1)
    assert not math.isfinite(norm.item()) and math.isnan(norm.item()) == math.isnan(bad)
    outs = [torch.zeros_like(t) for t in g]
    clip_grads(g, 0.1, outs=outs)
    for a, o, r in zip(g, outs, ref):
        assert torch.equal(a.nan_to_num(7.0), r.nan_to_num(7.0))
        assert torch.equal(o.nan_to_num(7.0), r.nan_to_num(7.0))


def test_a_norm_past_float32():
    """Finite values whose norm float32 cannot hold: infinite as it is read,
    so the values stay."""
    g = [torch.full((100,), 3e38, device="cuda"), torch.ones(5, device="cuda", dtype=B)]
    ref = [t.clone() for t in g]
    assert clip_grads(g, 1.0).item() == math.inf
    assert all(torch.equal(a, r) for a, r in zip(g, ref))


def test_by_a_given_norm():
    g = make([(5000, F), (777, B)], seed=5)
    a, b = [t.clone() for t in g], [t.clone() for t in g]
    n = clip_grads(a, 3.0)
    m = clip_grads(b, 3.0, norm=grad_norm(b))
    assert torch.equal(n, m)
    # (the factor from the float32 norm, not the float64 one: one more rounding)
    assert ((a[0] - b[0]).abs() <= 2.0 ** -22 * a[0].abs()).all()
    assert ((a[1].float() - b[1].float()).abs() <= 2.0 ** -7 * a[1].float().abs()).all()
    joined = torch.tensor(1e3, device="cuda")  # a larger norm, as from other ranks
    clip_grads(g, 5.0, norm=joined)
    ref = make([(5000, F), (777, B)], seed=5)[0]
    assert ((g[0] - ref * 5e-3).abs() <= 2.0 ** -22 * g[0].abs()).all()


def test_side_stream_and_graph():
    sizes = [(40_000, F), (999, B), (123_457, F)]
    g = make(sizes, seed=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = [t.clone() for t in g]
    s.wait_stream(torch.cuda.current_stream())
    n = clip_grads(a, 1.0, stream=s)
    s.synchronize()
    b = [t.clone() for t in g]
    m = clip_grads(b, 1.0)
    assert torch.equal(n, m) and all(torch.equal(x, y) for x, y in zip(a, b))
    buf = [torch.zeros_like(t) for t in g]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip_grads(buf, 1.0)
    for k in range(4):
        new = make(sizes, seed=20 + k, scale=1.0 if k % 2 else 1e-6)
        for t, v in zip(buf, new):
            t.copy_(v)
        graph.replay()
        eager = clip_grads(new, 1.0)
        torch.cuda.synchronize()
        assert torch.equal(norm, eager)
        assert all(torch.equal(x, y) for x, y in zip(buf, new))


def test_refusals():
    g = torch.ones(64, device="cuda")
    for call in (lambda: clip_grads([g.half()], 1.0), lambda: clip_grads([g.cpu()], 1.0),
                 lambda: clip_grads([g], 1.0, outs=[]), lambda: clip_grads([g[::2]], 1.0),
                 lambda: clip_grads([g], 1.0, outs=[torch.empty(63, device="cuda")]),
                 lambda: clip_grads([g], 1.0, outs=[torch.empty(64, device="cuda", dtype=B)]),
                 lambda: clip_grads([g, g.cpu()], 1.0),
                 lambda: clip_grads([g], 1.0, norm=torch.ones(2, device="cuda")),
                 lambda: clip_grads([g], 1.0, norm=torch.ones(())),
                 lambda: grad_norm([g.double()])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: clip_grads([g], -1.0), lambda: clip_grads([g], math.nan),
                 lambda: clip_grads([g, g], 1.0), lambda: clip_grads([g[:40], g[30:]], 1.0),
                 lambda: clip_grads([g[:32]], 1.0, outs=[g[16:48]]),
                 lambda: clip_grads([g[1:], g[:1]], 1.0, norm=g[3])):
        with pytest.raises(P.PoetxError):
            call()
    assert torch.equal(g, torch.ones_like(g))
    assert grad_norm([g, g]).item() == math.sqrt(128.0) or \
        abs(grad_norm([g, g]).item() - math.sqrt(128.0)) <= 2.0 ** -23 * 12

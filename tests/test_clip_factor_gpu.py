"""Clipping where the factor max_norm / norm is far from 1. The factor keeps 48
bits as hi + lo, so a clipped value is off by its output rounding alone: half a
step of float32, 2^-24 relative or 2^-150 where the result is below 2^-126;
bfloat16 by way of float32, 2^-8 (1 + 2^-15) relative or, below 2^-126, half of
its step 2^-133 and of float32's. 2^-46 for the rest: lo is below 2^-24, its
rounding 2^-49 and that of v lo 2^-48 |v|, against a result of |v| / 2 at least,
and the float64 steps."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here is gpu-marked
    pytest.skip("no GPU", allow_module_level=True)

from orthogonal_equivalence_amd.grads import clip_grads, grad_norm  # noqa: E402

REL = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8 * (1 + 2.0 ** -15)}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134 + 2.0 ** -150}


def check(g, out, factor):
    want = g.double() * factor
    tol = (REL[g.dtype] + 2.0 ** -46) * want.abs() + TINY[g.dtype]
    worst = ((out.double() - want).abs() / tol).max().item()
    print(f"    {g.dtype} factor {factor:.3e}: worst error / tolerance {worst:.4f}", flush=True)
    assert worst <= 1.0


# factors from 0.3 to below float32's smallest number
@pytest.mark.parametrize("scale,max_norm", [(1.0, 0.3), (1.0, 77.0), (1e20, 1e-3), (1e30, 1e-9),
                                            (1e33, 1e-8), (1e35, 1e-8), (1e36, 1e-9), (1e36, 1e-7)])
@pytest.mark.parametrize("given", [False, True], ids=["measured", "given"])
def test_factor(scale, max_norm, given):
    gen = torch.Generator(device="cuda").manual_seed(2)
    # whole chunks, a cut one, and values off the vector boundary
    flat = torch.randn(40_000, generator=gen, device="cuda") * scale
    grads = [flat[:20_001], flat[20_005:39_999], (flat[:9_001] * 0.5).bfloat16()]
    norm64 = sum(g.double().square().sum() for g in grads).sqrt().item()
    outs = [torch.full_like(g, 3.0) for g in grads]
    norm = grad_norm(grads) if given else None
    measured = clip_grads(grads, max_norm, outs, norm=norm)
    # (max_norm as the call takes it, in float32; a given norm is float32 too)
    limit = torch.tensor(max_norm, dtype=torch.float32).double().item()
    by = measured.double().item() if given else norm64
    assert by > limit
    for g, out in zip(grads, outs):
        check(g, out, limit / by)
    clip_grads(grads, max_norm, norm=norm)  # in place
    assert all(torch.equal(g, o) for g, o in zip(grads, outs))


@pytest.mark.parametrize("max_norm", [0.5, 0.3, 0.1, 1e-30])
def test_infinities_under_a_finite_given_norm_stay(max_norm):
    inf = float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        g = torch.arange(1, 9001, device="cuda").remainder(97).add(1).to(dtype)
        g[5], g[8999] = inf, -inf
        out = torch.zeros_like(g)
        norm = torch.ones((), device="cuda")
        clip_grads([g], max_norm, [out], norm=norm)
        assert out[5] == inf and out[8999] == -inf
        finite = torch.isfinite(g)
        check(g[finite], out[finite], torch.tensor(max_norm, dtype=torch.float32).double().item())


def test_factors_of_one_and_zero_and_powers_of_two_are_exact():
    gen = torch.Generator(device="cuda").manual_seed(3)
    for dtype in (torch.float32, torch.bfloat16):
        g = torch.randn(9001, generator=gen, device="cuda").to(dtype)
        for norm, factor in ((1.0, 1.0), (4.0, 0.25), (2.0 ** 40, 2.0 ** -40)):
            out = torch.zeros_like(g)
            clip_grads([g], 1.0, [out], norm=torch.tensor(norm, device="cuda"))
            assert torch.equal(out, g * factor)
        out = torch.full_like(g, 7.0)
        clip_grads([g], 0.0, [out], norm=torch.ones((), device="cuda"))
        assert not out.any()

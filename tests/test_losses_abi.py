"""The C ABI of the losses over a vocabulary without a GPU: sizes and every
host-detectable error (validation runs before any HIP call)."""
import pytest

P = pytest.importorskip("orthogonal_equivalence_amd.poetx",
                        reason="libpoetx.so not built (run the build first)")

A = 1 << 32  # a fake aligned address; validation never dereferences it


@pytest.fixture(autouse=True)
def _cpu_only():
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-validation tests use fake device addresses; run them without a GPU")


SMALL = dict(tokens=16, d=64, vocab=101, act=P.POETX_BF16, top=0, teacher=0, temperature=1.0)
LIST = dict(top=4, teacher=P.POETX_BF16, temperature=2.0)


def desc(**over):
    k = dict(SMALL, **over)
    d = P.make_vocab_desc(*(k[n] for n in ("tokens", "d", "vocab", "act", "top", "teacher",
                                           "temperature")))
    d.flags, d.reserved = k.get("flags", 0), k.get("reserved", 0)
    return d


def ce_fwd(over=(), **d):
    a = dict(x=A, W=2 * A, ids=3 * A, loss=4 * A, lse=5 * A, ws=7 * A, n=1 << 40)
    a.update(over)
    return P._lib.poetx_cross_entropy_fwd(desc(**d), a["x"], a["W"], a["ids"], a["loss"], a["lse"],
                                          a["ws"], a["n"], None)


def ce_bwd(over=(), **d):
    a = dict(g=A, g_lse=2 * A, x=3 * A, W=4 * A, ids=5 * A, lse=6 * A, g_x=7 * A, g_W=8 * A,
             ws=9 * A, n=1 << 40)
    a.update(over)
    return P._lib.poetx_cross_entropy_bwd(desc(**d), a["g"], a["g_lse"], a["x"], a["W"], a["ids"],
                                          a["lse"], a["g_x"], a["g_W"], a["ws"], a["n"], None)


def kd_fwd(over=(), **d):
    a = dict(x=A, W=2 * A, ids=3 * A, teacher=4 * A, loss=5 * A, lse=6 * A, z=7 * A, ws=8 * A,
             n=1 << 40)
    a.update(over)
    return P._lib.poetx_distill_fwd(desc(**{**LIST, **d}), a["x"], a["W"], a["ids"], a["teacher"],
                                    a["loss"], a["lse"], a["z"], a["ws"], a["n"], None)


def kd_bwd(over=(), **d):
    a = dict(g=A, x=2 * A, W=3 * A, ids=4 * A, teacher=5 * A, lse=6 * A, z=7 * A, g_x=8 * A,
             g_W=9 * A, ws=10 * A, n=1 << 40)
    a.update(over)
    return P._lib.poetx_distill_bwd(desc(**{**LIST, **d}), a["g"], a["x"], a["W"], a["ids"],
                                    a["teacher"], a["lse"], a["z"], a["g_x"], a["g_W"], a["ws"],
                                    a["n"], None)


CALLS = [ce_fwd, ce_bwd, kd_fwd, kd_bwd]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad,status", [
    (dict(act=2), P.POETX_ERR_DTYPE), (dict(act=-1), P.POETX_ERR_DTYPE),
    (dict(tokens=0), P.POETX_ERR_SHAPE), (dict(tokens=-1), P.POETX_ERR_SHAPE),
    (dict(tokens=(1 << 24) + 1), P.POETX_ERR_SHAPE), (dict(tokens=1 << 62), P.POETX_ERR_SHAPE),
    (dict(d=0), P.POETX_ERR_SHAPE), (dict(d=(1 << 22) + 8), P.POETX_ERR_SHAPE),
    (dict(vocab=0), P.POETX_ERR_SHAPE), (dict(vocab=(1 << 22) + 1), P.POETX_ERR_SHAPE),
    (dict(vocab=1 << 22, d=(1 << 13) + 8), P.POETX_ERR_SHAPE),
    (dict(tokens=1 << 24, d=(1 << 11) + 8), P.POETX_ERR_SHAPE),
    (dict(top=-1), P.POETX_ERR_SHAPE), (dict(top=1025), P.POETX_ERR_SHAPE),
    (dict(flags=1), P.POETX_ERR_SHAPE), (dict(reserved=1), P.POETX_ERR_SHAPE),
    (dict(d=60), P.POETX_ERR_ALIGN), (dict(act=P.POETX_F32, d=66), P.POETX_ERR_ALIGN),
])
def test_bad_descriptors(call, bad, status):
    assert call(**bad) == status
    for size in (P.poetx_vocab_fwd_workspace_size, P.poetx_vocab_bwd_workspace_size):
        assert size(desc(**bad)) == 0


@pytest.mark.parametrize("call", [kd_fwd, kd_bwd])
def test_bad_teachers(call):
    nan, inf = float("nan"), float("inf")
    for t in (0.0, -1.0, nan, inf, 1e-7, 1e7):
        assert call(temperature=t) == P.POETX_ERR_SHAPE, t
    assert call(teacher=2) == call(teacher=-1) == P.POETX_ERR_DTYPE
    assert call(top=0, teacher=0, temperature=1.0) == P.POETX_ERR_SHAPE


@pytest.mark.parametrize("call", [ce_fwd, ce_bwd])
def test_cross_entropy_takes_no_teacher(call):
    assert call(top=1) == P.POETX_ERR_SHAPE
    assert call(teacher=1) == call(temperature=2.0) == P.POETX_ERR_SHAPE


def test_null_pointers():
    for call, names in ((ce_fwd, ("x", "W", "ids", "loss", "lse")),
                        (ce_bwd, ("g", "x", "W", "ids", "lse")),
                        (kd_fwd, ("x", "W", "ids", "teacher", "loss", "lse", "z")),
                        (kd_bwd, ("g", "x", "W", "ids", "teacher", "lse", "z"))):
        for n in names:
            assert call({n: None}) == P.POETX_ERR_NULL, (call, n)
        assert call({"ws": None}) == P.POETX_ERR_WORKSPACE
    for call in (ce_bwd, kd_bwd):
        assert call({"g_x": None, "g_W": None}) == P.POETX_ERR_NULL
    assert P._lib.poetx_cross_entropy_fwd(None, A, A, A, A, A, A, 1, None) == P.POETX_ERR_NULL
    assert P.poetx_vocab_fwd_workspace_size(None) == 0


def test_alignment():
    for call, names in ((ce_fwd, ("x", "W", "ids", "loss", "lse", "ws")),
                        (ce_bwd, ("g", "g_lse", "x", "W", "ids", "lse", "g_x", "g_W", "ws")),
                        (kd_fwd, ("x", "W", "ids", "teacher", "loss", "lse", "z", "ws")),
                        (kd_bwd, ("g", "x", "W", "ids", "teacher", "lse", "z", "g_x", "g_W", "ws"))):
        for n in names:
            assert call({n: 64 * A + 1}) == P.POETX_ERR_ALIGN, (call, n)
    assert ce_fwd({"ids": 64 * A + 4}) == P.POETX_ERR_ALIGN


def test_workspace_too_small():
    for call, d, size in ((ce_fwd, desc(), P.poetx_vocab_fwd_workspace_size),
                          (ce_bwd, desc(), P.poetx_vocab_bwd_workspace_size),
                          (kd_fwd, desc(**LIST), P.poetx_vocab_fwd_workspace_size),
                          (kd_bwd, desc(**LIST), P.poetx_vocab_bwd_workspace_size)):
        assert size(d) > 0
        assert call({"n": size(d) - 1}) == P.POETX_ERR_WORKSPACE


def test_overlaps():
    for call, outs, ins in (
            (ce_fwd, ("loss", "lse", "ws"), ("x", "W", "ids")),
            (ce_bwd, ("g_x", "g_W", "ws"), ("g", "g_lse", "x", "W", "ids", "lse")),
            (kd_fwd, ("loss", "lse", "z", "ws"), ("x", "W", "ids", "teacher")),
            (kd_bwd, ("g_x", "g_W", "ws"), ("g", "x", "W", "ids", "teacher", "lse", "z"))):
        for i, o in enumerate(outs):
            for other in ins + outs[i + 1:]:
                assert call({o: 50 * A, other: 50 * A}) == P.POETX_ERR_ALIAS, (call, o, other)


def test_workspaces_stay_bounded():
    """Neither direction holds the logits: what they take beyond a copy of x and
    a float32 gradient of it is bounded, but for 256 columns (or rows) at the least."""
    for tokens, d, vocab in ((8192, 4096, 131072), (65536, 1024, 262144), (100, 512, 1 << 22),
                             (1 << 20, 64, 1 << 20)):
        for act, es in ((P.POETX_BF16, 2), (P.POETX_F32, 4)):
            k = desc(tokens=tokens, d=d, vocab=vocab, act=act)
            fwd, bwd = P.poetx_vocab_fwd_workspace_size(k), P.poetx_vocab_bwd_workspace_size(k)
            assert 0 < fwd <= (130 << 20) + 4 * tokens + 256 * vocab // 16 * 8
            piece = max(516 << 20, tokens * 256 * es)
            assert 0 < bwd <= piece + tokens * (d * (es + 4) + 20) + (256 << 20), (tokens, act)


def test_python_refusals():
    """The binding's own checks, on CPU tensors and wrong types and shapes."""
    import torch

    from orthogonal_equivalence_amd import losses as L
    x, W, t = torch.zeros(4, 8), torch.zeros(9, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        L.cross_entropy_forward(x, W, t)
    with pytest.raises(ValueError, match="expected float32 or bfloat16"):
        L.cross_entropy_forward(x.half(), W.half(), t)
    with pytest.raises(ValueError, match="GPU"):
        L.distill_forward(x, W, t[:, None], x[:, :1])

"""The C ABI of the dense linear and of gradient clipping without a GPU:
sizes and every host-detectable error (validation runs before any HIP call)."""
import array
import ctypes

import pytest

P = pytest.importorskip("orthogonal_equivalence_amd.poetx",
                        reason="libpoetx.so not built (run the build first)")

A = 1 << 20  # a fake 16-byte aligned address; validation never dereferences it


@pytest.fixture(autouse=True)
def _cpu_only():
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-validation tests use fake device addresses; run them without a GPU")


SMALL = dict(tokens=16, d_in=64, d_out=64, act=P.POETX_BF16, activation=P.POETX_ACT_SILU,
             w_scale=None)


def desc(**over):
    k = dict(SMALL, **over)
    d = P.make_dense_desc(k["tokens"], k["d_in"], k["d_out"], k["act"], k["activation"],
                          k["w_scale"])
    d.flags, d.reserved = k.get("flags", 0), k.get("reserved", 0)
    return d


def fwd(d, **over):
    a = dict(x=A, W=2 * A, bias=3 * A, residual=4 * A, y=5 * A, u=6 * A, ws=7 * A, ws_bytes=1 << 40)
    a.update(over)
    return P._lib.poetx_dense_fwd(d, a["x"], a["W"], a["bias"], a["residual"], a["y"], a["u"],
                                  a["ws"], a["ws_bytes"], None)


def bwd(d, **over):
    a = dict(g_y=A, x=2 * A, W=3 * A, u=4 * A, g_x=5 * A, g_W=6 * A, g_b=7 * A, ws=8 * A,
             ws_bytes=1 << 40)
    a.update(over)
    return P._lib.poetx_dense_bwd(d, a["g_y"], a["x"], a["W"], a["u"], a["g_x"], a["g_W"],
                                  a["g_b"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("bad,status", [
    (dict(act=2), P.POETX_ERR_DTYPE), (dict(act=-1), P.POETX_ERR_DTYPE),
    (dict(tokens=0), P.POETX_ERR_SHAPE), (dict(tokens=-1), P.POETX_ERR_SHAPE),
    (dict(tokens=1 << 31), P.POETX_ERR_SHAPE), (dict(d_in=0), P.POETX_ERR_SHAPE),
    (dict(d_out=-8), P.POETX_ERR_SHAPE), (dict(d_in=(1 << 22) + 8), P.POETX_ERR_SHAPE),
    (dict(d_out=(1 << 22) + 8), P.POETX_ERR_SHAPE),
    (dict(tokens=(1 << 31) - 1, d_out=1 << 22), P.POETX_ERR_SHAPE),
    (dict(activation=-1), P.POETX_ERR_SHAPE), (dict(activation=5), P.POETX_ERR_SHAPE),
    (dict(flags=1), P.POETX_ERR_SHAPE), (dict(reserved=1), P.POETX_ERR_SHAPE),
    (dict(d_in=60), P.POETX_ERR_ALIGN), (dict(d_out=36), P.POETX_ERR_ALIGN),
    (dict(act=P.POETX_F32, d_in=66), P.POETX_ERR_ALIGN),
    (dict(act=P.POETX_F32, d_in=68, w_scale=A), P.POETX_ERR_ALIGN),
    (dict(w_scale=A + 4), P.POETX_ERR_ALIGN),
])
def test_bad_descriptors(call, bad, status):
    assert call(desc(**bad)) == status
    assert P.poetx_dense_fwd_workspace_size(desc(**bad)) == 0
    assert P.poetx_dense_bwd_workspace_size(desc(**bad)) == 0


def test_null_pointers():
    for k in ("x", "W", "y"):
        assert fwd(desc(), **{k: None}) == P.POETX_ERR_NULL, k
    for k in ("g_y", "x", "W", "u"):
        assert bwd(desc(), **{k: None}) == P.POETX_ERR_NULL, k
    assert bwd(desc(), g_x=None, g_W=None, g_b=None) == P.POETX_ERR_NULL
    assert P._lib.poetx_dense_fwd(None, A, A, A, A, A, A, A, 1, None) == P.POETX_ERR_NULL
    assert P._lib.poetx_dense_bwd(None, A, A, A, A, A, A, A, A, 1, None) == P.POETX_ERR_NULL


def test_alignment_of_pointers():
    for k in ("x", "W", "bias", "residual", "y", "u"):
        assert fwd(desc(), **{k: 9 * A + 8}) == P.POETX_ERR_ALIGN, k
    for k in ("g_y", "x", "W", "u", "g_x", "g_W", "g_b", "ws"):
        assert bwd(desc(), **{k: 9 * A + 8}) == P.POETX_ERR_ALIGN, k


def test_workspace():
    # a long reduction of few tiles, and INT8 codes whose rows are not whole 16
    # bytes (widened into it), need one in the forward
    for d in (desc(tokens=200, d_in=4096), desc(tokens=200, d_in=72, w_scale=A * 16)):
        need = P.poetx_dense_fwd_workspace_size(d)
        assert need > 0
        assert fwd(d, ws=None) == P.POETX_ERR_WORKSPACE
        assert fwd(d, ws_bytes=need - 1) == P.POETX_ERR_WORKSPACE
        assert fwd(d, ws=7 * A + 8) == P.POETX_ERR_ALIGN
    need = P.poetx_dense_bwd_workspace_size(desc())
    assert bwd(desc(), ws=None) == P.POETX_ERR_WORKSPACE
    assert bwd(desc(), ws_bytes=need - 1) == P.POETX_ERR_WORKSPACE


def test_aliases():
    d = desc()
    assert fwd(d, y=A) == P.POETX_ERR_ALIAS              # y over x
    assert fwd(d, y=4 * A) == P.POETX_ERR_ALIAS          # y over the residual
    assert fwd(d, u=5 * A + 16) == P.POETX_ERR_ALIAS     # u over y
    assert fwd(d, u=2 * A) == P.POETX_ERR_ALIAS          # u over W
    q = desc(tokens=200, d_in=4096)
    assert fwd(q, ws=A) == P.POETX_ERR_ALIAS             # the workspace over x
    for out in ("g_x", "g_W", "g_b"):
        for at in (A, 2 * A, 3 * A, 4 * A):
            assert bwd(d, **{out: at}) == P.POETX_ERR_ALIAS, (out, at)
    assert bwd(d, g_W=5 * A) == P.POETX_ERR_ALIAS
    assert bwd(d, ws=5 * A) == P.POETX_ERR_ALIAS


def test_what_is_not_read_may_be_anything():
    """An unused u, x or W over an output, or misaligned, is no error: the call
    gets as far as its workspace."""
    none = desc(activation=P.POETX_ACT_NONE)
    for d, over in ((none, dict(u=5 * A)), (none, dict(u=3)), (desc(), dict(g_W=None, x=5 * A)),
                    (desc(), dict(g_x=None, W=6 * A + 1))):
        assert bwd(d, ws=None, **over) == P.POETX_ERR_WORKSPACE


def test_codes_have_no_gradient():
    assert bwd(desc(w_scale=A * 16)) == P.POETX_ERR_DTYPE


def test_workspace_sizes_of_large_layers():
    d = desc(tokens=8192, d_in=4096, d_out=14336)
    assert 8192 * 14336 * 2 <= P.poetx_dense_bwd_workspace_size(d) < 1 << 30
    d = desc(tokens=1 << 20, d_in=1 << 15, d_out=1 << 15)
    assert P.poetx_dense_bwd_workspace_size(d) >= (1 << 20) * (1 << 15) * 2


# ------------------------------------------------------------- gradient lists
def items(*rows):
    return array.array("Q", [v for r in rows for v in r])


def norm(rows, count=None, out=9 * A, ws=10 * A, ws_bytes=1 << 20):
    t = items(*rows)
    return P._lib.poetx_grad_norm(t.buffer_info()[0] if t else None,
                                  len(rows) if count is None else count, out, ws, ws_bytes, None)


def clip(rows, count=None, max_norm=1.0, out=9 * A, ws=10 * A, ws_bytes=1 << 20):
    t = items(*rows)
    return P._lib.poetx_grad_clip(t.buffer_info()[0] if t else None,
                                  len(rows) if count is None else count, max_norm, out, ws,
                                  ws_bytes, None)


def scale(rows, max_norm=1.0, norm_in=9 * A):
    t = items(*rows)
    return P._lib.poetx_grad_scale(t.buffer_info()[0], len(rows), max_norm, norm_in, None)


def test_grad_records_match_the_struct():
    assert ctypes.sizeof(P.GradTensor) == 32
    t = items((A, 2 * A, 100, P.POETX_BF16))
    g = P.GradTensor.from_buffer(t)
    assert (g.grad, g.out, g.n, g.dtype, g.reserved) == (A, 2 * A, 100, P.POETX_BF16, 0)


@pytest.mark.parametrize("row,status", [
    ((A, A, 100, 2), P.POETX_ERR_DTYPE), ((A, A, 100, 1 << 32), P.POETX_ERR_SHAPE),
    ((A, A, (1 << 64) - 1, 0), P.POETX_ERR_SHAPE), ((A, A, 1 << 50, 0), P.POETX_ERR_SHAPE),
    ((0, 0, 100, 0), P.POETX_ERR_NULL), ((A + 2, A + 2, 100, 0), P.POETX_ERR_ALIGN),
    ((A + 1, A + 1, 100, 1), P.POETX_ERR_ALIGN),
])
def test_bad_tensors(row, status):
    good = (20 * A, 20 * A, 10, 0)
    for call in (norm, clip, scale):
        assert call([good, row]) == status


def test_bad_list_arguments():
    good = (20 * A, 20 * A, 10, 0)
    assert norm([good], count=-1) == P.POETX_ERR_SHAPE and clip([good], count=-1) == P.POETX_ERR_SHAPE
    assert P._lib.poetx_grad_norm(None, 1, 9 * A, 10 * A, 1 << 20, None) == P.POETX_ERR_NULL
    assert norm([good], out=None) == P.POETX_ERR_NULL and clip([good], out=None) == P.POETX_ERR_NULL
    assert scale([good], norm_in=None) == P.POETX_ERR_NULL
    assert clip([(20 * A, 0, 10, 0)]) == P.POETX_ERR_NULL
    assert norm([good], out=9 * A + 2) == P.POETX_ERR_ALIGN
    assert norm([good], ws=None) == P.POETX_ERR_WORKSPACE
    assert norm([good], ws=10 * A + 8) == P.POETX_ERR_ALIGN
    need = P.poetx_grad_workspace_size(1)
    assert need > 0 and norm([good], ws_bytes=need - 1) == P.POETX_ERR_WORKSPACE
    assert P.poetx_grad_workspace_size(-1) == 0 and P.poetx_grad_workspace_size(0) > 0
    for bad in (-1.0, float("nan"), float("-inf")):
        assert clip([good], max_norm=bad) == P.POETX_ERR_SHAPE
        assert scale([good], max_norm=bad) == P.POETX_ERR_SHAPE


def test_list_aliases():
    n = 1000  # 4000 bytes in float32
    a, b = 20 * A, 30 * A
    assert clip([(a, b, n, 0), (a + 4000, b + 3996, n, 0)]) == P.POETX_ERR_ALIAS  # outs overlap
    assert clip([(a, a, n, 0), (a, a, n, 0)]) == P.POETX_ERR_ALIAS               # listed twice
    assert clip([(a, a + 16, n, 0)]) == P.POETX_ERR_ALIAS                        # shifted
    assert clip([(a, b, n, 0), (b + 100, 40 * A, n, 0)]) == P.POETX_ERR_ALIAS    # over a gradient
    assert clip([(a, a, n, 0), (a + 3000, b, 10, 0)]) == P.POETX_ERR_ALIAS
    assert clip([(a, a, n, 0)], out=a + 40) == P.POETX_ERR_ALIAS                 # norm inside
    assert norm([(a, a, n, 0)], out=a + 40) == P.POETX_ERR_ALIAS
    assert norm([(a, a, n, 0)], ws=a) == P.POETX_ERR_ALIAS
    assert norm([(a, a, n, 0)], out=10 * A + 8) == P.POETX_ERR_ALIAS             # norm in the ws
    assert scale([(a, a, n, 0)], norm_in=a + 40) == P.POETX_ERR_ALIAS
    # a contained range that starts before the writer's end, far down the list
    rows = [(a + 8000 * i, a + 8000 * i, n, 0) for i in range(200)]
    assert clip(rows + [(a + 8000 * 150 + 400, b, 4, 0)]) == P.POETX_ERR_ALIAS

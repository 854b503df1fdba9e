"""What the dense linear's calls launch, from the sizes alone (CPU): the plans of
csrc/dense_plan.cpp, compiled with the host compiler into a program that prints
them, and the refusals of the C ABI that follow from them."""
import functools
import os
import random
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "orthogonal_equivalence_amd", "csrc")

# reads lines "dtype int8 tokens d_in d_out" and prints the choices
PROGRAM = r"""
#include <cstdio>
#include "dense_plan.h"
using namespace poetx;
int main() {
  int t, int8;
  long long m, n, k;
  while (scanf("%d %d %lld %lld %lld", &t, &int8, &m, &n, &k) == 5) {
    const DType d = static_cast<DType>(t);
    const FwdChoice f = choose_fwd(d, int8, m, n, k);
    const BwdChoice b = choose_bwd(d, int8, m, n, k);
    printf("%d %d %d %d %d %d %d %d %d %d %d %d %d %d %d %d %d %d %d\n", f.launchable(),
           b.gx_launchable(), b.gw_launchable(), f.stream, f.dense, f.widen, f.w_tiled, f.tile.shape, f.tile.nsplit, b.dense, b.paired,
           b.gx.shape, b.gx.nsplit, b.gw.shape, b.gw.nsplit, b.pair.gx.shape, b.pair.gx.nsplit,
           b.pair.gw.shape, b.pair.gw.nsplit);
  }
}
"""
FIELDS = ("y_fits", "gx_fits", "gw_fits", "stream", "dense", "widen", "w_tiled", "shape", "split", "b_dense", "paired",
          "gx_shape", "gx_split", "gw_shape", "gw_split", "px_shape", "px_split", "pw_shape",
          "pw_split")
F32, BF16 = 0, 1
# the tile shapes of the plans: rows, columns, threads
SHAPES = {BF16: ((256, 128, 512), (128, 128, 512), (128, 64, 512), (64, 64, 256), (32, 64, 256),
                 (128, 64, 512)),
          F32: ((64, 64, 256), (32, 64, 256))}


@functools.lru_cache(maxsize=None)
def _program():
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the HIP headers")
    folder = tempfile.mkdtemp(prefix="dense_plan_")
    src, exe = os.path.join(folder, "main.cpp"), os.path.join(folder, "plans")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), src,
                    os.path.join(CSRC, "dense_plan.cpp"), "-o", exe], check=True)
    return exe


def plans(cases):
    """The choices for each (dtype, int8, tokens, d_in, d_out), as dicts."""
    text = "".join("%d %d %d %d %d\n" % c for c in cases)
    out = subprocess.run([_program()], input=text, capture_output=True, text=True, check=True).stdout
    rows = [dict(zip(FIELDS, map(int, line.split()))) for line in out.splitlines()]
    assert len(rows) == len(cases)
    return rows


def work_items(dtype, shape, M, N, split=1, pad=0):
    bm, bn, threads = SHAPES[dtype][shape]
    return (-(-M // bm) * -(-N // bn) * split + pad) * threads


def test_every_chosen_launch_fits():
    """tiles x threads below 2^32, what HIP takes along one dimension, over the
    whole range that the descriptor allows, also where no memory holds it."""
    rng = random.Random(1)
    cases = [(t, 0, tokens, n, k) for t in (F32, BF16)
             for tokens in (1 << 28, (1 << 29) - 64, (1 << 29) - 63, 1 << 29, (1 << 30) - 64,
                            (1 << 30) - 63, 1 << 30)
             for n in (8, 64, 72, 128) for k in (8, 64, 72, 128)]
    cases += [(t, 0, tokens, n, k) for t in (F32, BF16) for tokens in (9, 5000)
              for n, k in ((1 << 22, 1 << 22), (1 << 22, 1 << 14), (1 << 14, 1 << 22))]
    for _ in range(4000):
        n, k = (8 * rng.randint(1, 1 << rng.randint(0, 19)) for _ in range(2))
        cases.append((rng.randint(0, 1), 0, rng.randint(9, 1 << rng.randint(4, 30)), n, k))
    refused = 0
    for (t, _, m, n, k), p in zip(cases, plans(cases)):
        # an output is refused where no shape's tiles fit
        for fits, dense, shape, split, rows, cols in (
                (p["y_fits"], p["dense"], p["shape"], p["split"], m, k),
                (p["gx_fits"], p["b_dense"], p["gx_shape"], p["gx_split"], m, n),
                (p["gw_fits"], 0, p["gw_shape"], p["gw_split"], k, n)):
            if dense:
                assert fits
            elif fits:
                assert split >= 1 and work_items(t, shape, rows, cols) < 1 << 32
            else:
                refused += 1
                assert all(work_items(t, i, rows, cols) >= 1 << 32 for i in range(len(SHAPES[t])))
        if p["paired"]:
            assert p["px_shape"] == p["pw_shape"] and p["px_split"] >= 1 and p["pw_split"] >= 1
            assert work_items(t, p["px_shape"], m, n, p["px_split"], 7) + \
                work_items(t, p["pw_shape"], k, n, p["pw_split"]) < 1 << 32
    assert refused > 20


def test_products_past_one_launch_are_refused():
    """Before anything is enqueued, and only where that output is asked for."""
    P = pytest.importorskip("orthogonal_equivalence_amd.poetx")
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-validation tests use fake device addresses; run them without a GPU")
    A = 1 << 44

    def status(tokens, d_in, d_out, act):
        """The forward's status, the backward's of g_x, of g_W and of g_bias alone.
        (Validation ends at the aliased y, or at the missing workspace: nothing is
        launched on these addresses.)"""
        d = P.make_dense_desc(tokens, d_in, d_out, act, P.POETX_ACT_RELU)
        assert P.poetx_dense_bwd_workspace_size(d) > 0
        fwd = P._lib.poetx_dense_fwd(d, A, 2 * A, None, None, A, None, 4 * A, 1 << 43, None)
        return fwd, *(P._lib.poetx_dense_bwd(d, A, 2 * A, 3 * A, 4 * A, *outs, None, 0, None)
                      for outs in ((5 * A, None, None), (None, 5 * A, None), (None, None, 5 * A)))

    # past validation, and refused
    y, b, no = P.POETX_ERR_ALIAS, P.POETX_ERR_WORKSPACE, P.POETX_ERR_SHAPE
    for tokens, d_in, d_out, want in (
            (1 << 30, 8, 8, (no, no, b, b)), ((1 << 30) - 64, 8, 8, (y, b, b, b)),
            (1 << 29, 8, 72, (no, b, b, b)), (1 << 29, 72, 8, (y, no, b, b)),
            ((1 << 29) - 64, 72, 72, (y, b, b, b)), (9, 1 << 22, 1 << 14, (y, b, no, b))):
        assert status(tokens, d_in, d_out, P.POETX_F32) == want, (tokens, d_in, d_out)
        assert status(tokens, d_in, d_out, P.POETX_BF16) == (y, b, b, b), (tokens, d_in, d_out)

"""What the losses over a vocabulary launch, from the sizes alone (CPU): the plans of
csrc/vocab_plan.cpp, compiled with the host compiler into a program that prints
them; the cases of vocab_cases.py reach every variant that they choose."""
import functools
import math
import os
import random
import shutil
import subprocess
import tempfile

import pytest

from tests.vocab_cases import CASES, LISTED

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "orthogonal_equivalence_amd", "csrc")

# reads lines "dtype tokens d vocab top weight" and prints the forward's choices and
# the backward's (weight: of both gradients), piece by piece
PROGRAM = r"""
#include <cstdio>
#include <algorithm>
#include "vocab_plan.h"
using namespace poetx;
int main() {
  int t, top, weight;
  long long m, d, n;
  while (scanf("%d %lld %lld %lld %d %d", &t, &m, &d, &n, &top, &weight) == 6) {
    const VocabSizes v{static_cast<DType>(t), m, d, n, top};
    const VocabFwdPlan f = plan_vocab_fwd(v);
    const VocabBwdPlan b = plan_vocab_bwd(v, weight != 0);
    printf("%lld %d %d %lld %d %d %zu %d %lld %lld %lld %d %d %d %zu", (long long)f.cols.dense, f.cols.tile.shape,
           f.cols.tile.nsplit, (long long)f.rows, f.copied, f.cells, f.total, b.dense,
           (long long)b.padded, (long long)b.piece, (long long)b.ldg, b.few, b.splits, b.kchunk, b.total);
    for (long long c = 0; c < n; c += b.piece) {
      const long long cols = std::min<long long>(b.piece, n - c);
      const VocabColumns k = plan_vocab_columns(v, b, cols);
      const VocabProducts p = plan_vocab_products(v, cols);
      printf(" %lld %lld %d %d %d %d %d %d %d %d %d %d %d", cols, (long long)k.dense, k.tile.shape, k.tile.nsplit,
             p.gx.shape, p.gx.nsplit, p.gw.shape, p.gw.nsplit, p.paired, p.pair.gx.shape,
             p.pair.gx.nsplit, p.pair.gw.nsplit, p.few);
    }
    printf("\n");
  }
}
"""
FIELDS = ("dense", "shape", "split", "rows", "copied", "cells", "total", "b_dense", "padded",
          "piece", "ldg", "few", "splits", "kchunk", "b_total")
PIECE = ("cols", "dense", "shape", "split", "gx_shape", "gx_split", "gw_shape", "gw_split",
         "paired", "p_shape", "px_split", "pw_split", "p_few")
F32, BF16 = 0, 1


@functools.lru_cache(maxsize=None)
def _program():
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the HIP headers")
    folder = tempfile.mkdtemp(prefix="vocab_plan_")
    src, exe = os.path.join(folder, "main.cpp"), os.path.join(folder, "plans")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), src,
                    os.path.join(CSRC, "vocab_plan.cpp"), os.path.join(CSRC, "dense_plan.cpp"),
                    "-o", exe], check=True)
    return exe


def plans(cases, weight=1):
    """The choices for each (dtype, tokens, d, vocab, top), as dicts with a list
    of the backward's pieces."""
    text = "".join("%d %d %d %d %d %d\n" % (*c, weight) for c in cases)
    out = subprocess.run([_program()], input=text, capture_output=True, text=True, check=True).stdout
    rows = []
    for line in out.splitlines():
        v = list(map(int, line.split()))
        row, v = dict(zip(FIELDS, v)), v[len(FIELDS):]
        row["pieces"] = [dict(zip(PIECE, v[i:i + len(PIECE)])) for i in range(0, len(v), len(PIECE))]
        rows.append(row)
    assert len(rows) == len(cases)
    return rows


def parts(n):
    """Reductions cut into few or many parts are the same code."""
    return "whole" if n == 1 else "cut"


def variants(case, p):
    """The kernel variants of a case's forward and backward (both gradients)."""
    t, tokens, d, vocab, top = case
    got = set()
    if p["dense"]:
        got.add(("lse steps", d // 32 % 4))
        got.add(("lse", "listed" if top else "targets", "shifted" if tokens % 256 else "whole",
                 "padded" if p["dense"] % 256 else "full"))
    if p["dense"] < vocab:
        got.add(("lse tile", t, p["shape"], "beside" if p["dense"] else "alone"))
    got.add(("ranges", p["rows"] < tokens, p["dense"] > 0))
    if top:
        got.add(("listed", p["cells"], "dense" if p["dense"] else "tile", t))
        got.add(("listed gradient", t, p["b_dense"]))
    many = len(p["pieces"]) > 1
    for i, q in enumerate(p["pieces"]):
        if p["b_dense"]:
            if q["dense"]:
                got.add(("grad", "padded" if q["dense"] % 256 else "full"))
            whole = not many and p["splits"] == 1
            last = q["cols"] - (-(-q["cols"] // p["kchunk"]) - 1) * p["kchunk"]
            got.add(("gx", whole, q["cols"] % 32 != 0, min(last, p["kchunk"]) < 256))
            got.add(("gx steps", -(-last // 32) % 4 if last >= 256 else -(-last // 32)))
            steps = -(-tokens // 32)
            got.add(("gw steps", steps % 4 if steps >= 8 else steps))
            got.add(("grad steps", d // 32 % 4))
            got.add(("gx added", i > 0, d % 256 != 0, tokens % 256 != 0))
            got.add(("gw", d % 256 != 0, q["cols"] % 256 != 0, tokens % 32 != 0))
        else:
            got.add(("tile pieces", t, many))
        if q["dense"] < q["cols"]:
            got.add(("grad tile", t, q["shape"], p["b_dense"]))
        if p["b_dense"]:
            continue
        if p["few"]:
            es = 2 if t == BF16 else 4
            past = d * es % 128 == 0 and q["cols"] * d * es > 128 << 20
            got.add(("few", t, -(-tokens // (64 // es)), past))
        if p["few"] or not q["paired"]:
            got.add(("gx tile", t, q["gx_shape"], parts(q["gx_split"])))
            if not p["few"]:
                got.add(("gw tile", t, q["gw_shape"], parts(q["gw_split"])))
        else:
            got.add(("pair", t, q["p_shape"], parts(q["px_split"]), parts(q["pw_split"])))
    return got


def draw(rng):
    def size(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    t = rng.choice((F32, BF16, BF16))
    step = rng.choice((8, 8, 32, 256))
    d = max(step, size(8, 4096) // step * step)
    vocab = size(1, 131072)
    if rng.random() < 0.3:
        vocab = max(256, vocab // 256 * 256)
    tokens = max(1, min(size(1, 8192), (1 << 42) // (d * vocab)))
    return t, tokens, d, vocab, rng.choice((0, 0, size(1, 128)))


def test_cases_reach_every_variant():
    rng = random.Random(17)
    drawn = [draw(rng) for _ in range(20_000)]
    cases = [c + (0,) for c in CASES] + list(LISTED)
    reached = set()
    for c, p in zip(cases, plans(cases)):
        reached |= variants(c, p)
    missed = {}
    for c, p in zip(drawn, plans(drawn)):
        for v in variants(c, p) - reached:
            missed.setdefault(v, c)
    assert not missed, missed
    assert len(reached) > 60


def test_plans_hold_together():
    """Every product has a shape, ranges and pieces cover what they should, and the
    launchers' conditions hold, over the whole range that the descriptor allows."""
    rng = random.Random(3)
    cases = [draw(rng) for _ in range(5000)]
    for _ in range(2000):
        d = 8 * rng.randint(1, 1 << rng.randint(0, 19))
        most = (1 << 35) // d
        cases.append((rng.randint(0, 1), min(most, rng.randint(1, 1 << rng.randint(1, 24))), d,
                      min(most, rng.randint(1, 1 << rng.randint(1, 22))),
                      rng.choice((0, 1, rng.randint(1, 1024)))))
    cases += [(t, 1 << 24, 8, 1, 0) for t in (F32, BF16)] + [(t, 1, 8, 1 << 22, 1024) for t in (F32, BF16)]
    cases += [(t, 1 << 24, 1 << 11, 1 << 22, 1024) for t in (F32, BF16)]
    both = list(zip(cases, plans(cases))) + list(zip(cases, plans(cases, 0)))
    for (t, tokens, d, vocab, top), p in both:
        where = (t, tokens, d, vocab, top)
        assert 0 < p["total"] < 1 << 62 and 0 < p["b_total"] < 1 << 62, where
        assert p["dense"] == vocab or p["split"] == 1, where
        assert p["rows"] >= min(tokens, 256) and (p["rows"] == tokens or p["rows"] % 256 == 0), where
        if p["dense"]:
            assert t == BF16 and tokens >= 256 and p["rows"] >= 256 and d % 32 == 0 and d >= 256
            assert p["dense"] in (vocab, p["dense"] // 256 * 256) and p["copied"] == (p["dense"] % 256 > 0)
        assert p["ldg"] % 256 == 0 and p["ldg"] >= p["piece"], where
        assert sum(q["cols"] for q in p["pieces"]) == vocab
        for q in p["pieces"][:-1]:
            assert q["cols"] == p["piece"] and p["piece"] % 256 == 0
        for q in p["pieces"]:
            assert q["dense"] == q["cols"] or q["split"] == 1, where
            if p["b_dense"]:
                assert p["padded"] % 256 == 0 and p["padded"] >= tokens > 128
                assert p["kchunk"] % 32 == 0
                n = -(-q["cols"] // p["kchunk"])
                assert 1 <= n <= p["splits"], where
            else:
                assert q["gx_split"] >= 1 and q["gw_split"] >= 1, where
                if q["paired"]:
                    assert q["px_split"] >= 1 and q["pw_split"] >= 1, where
        assert not p["few"] or tokens <= (128 if t == BF16 else 64)

"""The elementwise scan's choice of slab, cluster and load (csrc/scan_plan.cuh, plain C++), asked without a GPU."""
import itertools
import os
import random
import shutil
import subprocess

import pytest

from chunkwise_linear_rnn_02_b200.build_lib import CSRC
from scan_shapes import SHAPES

PROGRAM = r"""
#include <stdio.h>
#include "scan_plan.cuh"
using namespace gla::scan;
template <bool BF16, int LOAD, bool COMP, bool BWD>
void ask(long long BH, int T, int D, const char* load) {
  const Plan p = choose<BF16, LOAD, COMP, BWD>(BH, T, D);
  auto print = [&](auto s) {
    printf("%s %s %d %s %d %lld %d %d %d %d %d %d %d\n", BF16 ? "bf16" : "f32", BWD ? "bwd" : "fwd", (int)COMP, load, p.lpr, p.cols,
           p.slabs, p.tiles, p.K, p.steps, s.STAGES, s.CW, s.MAXK);
  };
  if constexpr (!BWD)
    if (p.lpr == 32) return print(Shape<BF16, 32, BWD>());
  if (p.lpr == 16) return print(Shape<BF16, 16, BWD>());
  print(Shape<BF16, 8, BWD>());
}
template <bool BF16>
void all(long long BH, int T, int D) {
  const int es = BF16 ? 2 : 4;
  const char* load = by_tma(0, T, D, es) ? "tma" : fits(0, D, es, 2 * es) ? "pairs" : "single";
#define ASK(LOAD) \
  ask<BF16, LOAD, false, false>(BH, T, D, load), ask<BF16, LOAD, true, false>(BH, T, D, load), \
  ask<BF16, LOAD, false, true>(BH, T, D, load), ask<BF16, LOAD, true, true>(BH, T, D, load)
  if (by_tma(0, T, D, es)) ASK(kTma);
  else ASK(kByThread);
}
int main() {
  int bf16, T, D;
  long long BH;
  while (scanf("%d %lld %d %d", &bf16, &BH, &T, &D) == 4)
    if (bf16) all<true>(BH, T, D);
    else all<false>(BH, T, D);
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """plans(dtype, BH, T, D) of a list of calls: dicts, four a call."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    where = tmp_path_factory.mktemp("plan")
    (where / "ask.cpp").write_text(PROGRAM)
    exe = os.path.join(where, "ask")
    subprocess.run([cxx, "-std=c++17", "-O1", "-ftrapv", "-I", CSRC, str(where / "ask.cpp"), "-o", exe], check=True)

    def plans(calls):
        text = "".join(f"{int(t == 'bf16')} {bh} {n} {d}\n" for t, bh, n, d in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        names = ("dtype", "way", "complement", "load", "lpr", "cols", "slabs", "tiles", "K", "steps", "stages", "cw", "maxk")
        return [{n: v if n in ("dtype", "way", "load") else int(v) for n, v in zip(names, line.split())} for line in out.splitlines()]

    return plans


def test_the_tested_shapes_reach_every_kernel(ask):
    want = set()
    for t, way, comp, load, cluster in itertools.product(("bf16", "f32"), ("fwd", "bwd"), (0, 1), ("tma", "pairs", "single"), (0, 1)):
        widths = (16, 8) if way == "bwd" or (t == "f32" and load != "tma") else (32, 16, 8)
        want |= {(t, way, comp, load, w, cluster) for w in widths}
    got = set()
    for (t, load), shapes in SHAPES.items():
        for p in ask([(t, *s) for s in shapes]):
            assert p["load"] == load
            if p["steps"] > 2 * p["stages"]:
                got.add((t, p["way"], p["complement"], load, p["lpr"], int(p["K"] > 1)))
    assert got == want


def test_plans_cover_their_tokens_and_channels(ask):
    rng = random.Random(1)
    size = lambda most: max(1, round(most ** rng.random()))  # noqa: E731
    calls = [(rng.choice(("bf16", "f32")), size(4000), size(100000), size(8192)) for _ in range(3000)]
    calls += [(t, 1, n, d) for t in ("bf16", "f32") for n in (1, 130) for d in (2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 64)]
    calls += [(t, 2 ** 27, 1, 16) for t in ("bf16", "f32")] + [(t, 1, 2 ** 31 - 1, 1) for t in ("bf16", "f32")]
    for call, p in zip((c for c in calls for _ in range(4)), ask(calls)):
        _, BH, T, D = call
        assert (p["slabs"] - 1) * p["cw"] < D <= p["slabs"] * p["cw"], (call, p)
        assert p["cols"] == BH * p["slabs"] and p["cols"] * p["K"] < 2 ** 31, (call, p)
        assert 1 <= p["K"] <= p["maxk"] and p["K"] <= max(1, p["tiles"]), (call, p)
        assert (p["steps"] - 1) * p["K"] < p["tiles"] <= p["steps"] * p["K"], (call, p)

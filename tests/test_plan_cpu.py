"""The choice of tiles and splits of the linear layer's products (csrc/plan.hpp, host code without
HIP), compiled alone: it is valid for every size that a call takes, and the sizes that the GPU tests
run reach every kernel there is."""
import os
import random
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_compressed_backprop_amd", "csrc")

MAIN = r"""
#include <cstdio>
#include "plan.hpp"
int main() {
  for (const auto& s : instant::planning::SHAPES_FP32) printf("0 %d %d %d\n", s.wm, s.wn, s.ns);
  for (const auto& s : instant::planning::SHAPES_BF16) printf("1 %d %d %d\n", s.wm, s.wn, s.ns);
  printf("plans\n");
  int bf, m, n, k, heavy;
  while (scanf("%d %d %d %d %d", &bf, &m, &n, &k, &heavy) == 5) {
    const instant::Plan p = instant::plan(bf, m, n, k, heavy);
    printf("%d %d %d %d %d\n", p.wm, p.wn, p.ns, p.S, p.part);
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """rows (bfloat16, rows, columns, contraction, heavy) -> (shapes by type, [(wm, wn, ns, S, part)])"""
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, "-o", str(d / "plan"), str(d / "main.cpp")], check=True)

    def run(rows):
        text = "\n".join(" ".join(str(int(v)) for v in r) for r in rows)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        head, tail = out.split("plans\n")
        shapes = {0: set(), 1: set()}
        for line in head.splitlines():
            bf, *shape = map(int, line.split())
            shapes[bf].add(tuple(shape))
        plans = [tuple(map(int, line.split())) for line in tail.splitlines()]
        assert len(plans) == len(rows)
        return shapes, plans
    return run


def test_the_gpu_tests_sizes_reach_every_kernel(ask):
    """Every tile shape and ring depth of every product and type, whole and split."""
    import test_gpu_ops as G
    shapes, _ = ask([])
    for which in G.EVERY_TILE:
        kind, dtype = which
        bf = int(dtype == G.BF)
        found = set()
        for heavy in ((0, 1) if kind == "fwd" else (0,)):
            sizes = G.EVERY_TILE[which] + (G.LARGEST_SPLIT[dtype] if kind == "fwd" and not heavy else [])
            for p in ask([(bf, *s, heavy) for s in sizes])[1]:
                found.add((p[:3], p[3] > 1))
        assert found == {(s, split) for s in shapes[bf] for split in (False, True)}, which


def test_every_plan_is_valid(ask):
    """One of the compiled tiles, and a stage (128 bytes of the contraction) at least for every slice
    and partials for more than one, from the smallest sizes to the largest."""
    rng = random.Random(9)
    rows = [(bf, m, n, k, h) for bf in (0, 1) for h in (0, 1) for m in (1, 1 << 26) for n in (8, 1 << 18)
            for k in (8, 1 << 18)]
    rows += [(bf, n, k, m, 0) for bf in (0, 1) for m in (1, 1 << 26) for n in (8, 1 << 18) for k in (8, 1 << 18)]
    for _ in range(20000):
        rows.append((rng.randint(0, 1), int(2 ** rng.uniform(0, 20)), 8 * int(2 ** rng.uniform(0, 12)),
                     int(2 ** rng.uniform(0, 20)), rng.randint(0, 1)))
    shapes, plans = ask(rows)
    for r, (wm, wn, ns, S, part) in zip(rows, plans):
        stage = 64 if r[0] else 32
        assert (wm, wn, ns) in shapes[r[0]], r
        assert 1 <= S <= -(-r[3] // stage) and part == (S > 1), r

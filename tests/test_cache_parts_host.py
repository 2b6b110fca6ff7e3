"""How attention over the 4-bit cache cuts its work (Parts in csrc/sk_attn.cuh), on the CPU: sums
of 32 bits and beyond, which no test has the time to work off."""
import os
import subprocess

import numpy as np
import pytest

from conftest import ROOT

MAIN = r"""
#include <cstdio>
#include "sk_attn.cuh"
int main() {
  long long U, u;
  int G, c;
  while (scanf("%lld %d %d %lld", &U, &G, &c, &u) == 4) {
    const sk::Parts p(U, G);
    printf("%lld %d\n", p.start(c), p.of(u));
  }
}
"""


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    d = tmp_path_factory.mktemp("parts")
    (d / "parts.cu").write_text(MAIN)
    csrc, include = (os.path.join(ROOT, x) for x in ("nvfp4_sm_skinny_gb300/csrc", "include"))
    subprocess.run(["nvcc", "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", f"-I{csrc}", f"-I{include}",
                    "-o", str(d / "parts"), str(d / "parts.cu")], check=True)

    def run(cases):
        text = "".join("%d %d %d %d\n" % x for x in cases)
        out = subprocess.run([str(d / "parts")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return run


def test_parts_cover_the_work(parts):
    rng = np.random.default_rng(0)
    sums = [1, 2, 151, 152, 153, 1823, 1824, 1825, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 1, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 7,
            2 ** 43 + 12345, 2 ** 53 - 1]
    sums += [int(2 ** x) + int(y) for x, y in zip(rng.uniform(0, 54, 60), rng.integers(0, 100, 60))]
    cases = []
    for U in sums:
        for G in (1, 7, 152, 1824, 1920):
            cuts = [c * (U // G) + min(c, U % G) for c in range(G + 1)]
            for c in {0, 1, G - 1, G, min(U % G, G), *(int(x) for x in rng.integers(0, G + 1, 6))}:
                for u in {min(max(cuts[c] + e, 0), U - 1) for e in (-1, 0, 1)} | {int(rng.integers(0, U))}:
                    want = int(np.searchsorted(np.array(cuts[1:]), u, side="right"))
                    cases.append(((U, G, c, u), (cuts[c], want)))
    got = parts([x for x, _ in cases])
    assert len(got) == len(cases)
    for (x, want), have in zip(cases, got):
        assert want == have, (x, want, have)

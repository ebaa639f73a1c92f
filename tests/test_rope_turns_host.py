"""The turns per position that rotation tables are made from, against decimals of 80 digits."""
import math
import random
import subprocess
from decimal import Decimal, getcontext

import pytest

from quantized_paged_kv_kvq_gb300 import build

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include "rope_turns.h"
int main(int n, char** v) {  // rot_dim base kind factor original_len low high, again and again
  for (int k = 1; k + 6 < n; k += 7) {
    const kvq_rope_scaling sc = {atoi(v[k + 2]), atof(v[k + 3]), atof(v[k + 4]), atof(v[k + 5]), atof(v[k + 6]), 1.0};
    kvq::RopeTurns t;
    printf("%d", kvq::rope_turns(atoi(v[k]), atof(v[k + 1]), sc, &t) ? 1 : 0);
    for (int i = 0; i < atoi(v[k]) / 2; ++i) printf(" %llu", t.t[i]);
    printf("\n");
  }
  return 0;
}
"""
TURN = Decimal("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684")


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    d = tmp_path_factory.mktemp("turns")
    src, exe = d / "turns.cpp", d / "turns"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), "-std=c++17", "-Xcompiler", "-O2", "-I", build.CSRC, "-I", build.INCLUDE, str(src),
                    "-o", str(exe)], check=True)

    def run(cases):
        args = [repr(x) if isinstance(x, float) else str(x) for c in cases for x in c]
        out = subprocess.run([str(exe), *args], check=True, capture_output=True, text=True).stdout
        rows = [[int(x) for x in line.split()] for line in out.splitlines()]
        assert len(rows) == len(cases)
        return rows
    return run


def expected(rot, base, kind, factor, original, low, high):
    """theta_i / (2 pi) of every pair."""
    f, n, lo, hi = (Decimal(x) for x in (factor, original, low, high))
    out = []
    for i in range(rot // 2):
        theta = (Decimal(base).ln() * (-2 * i) / rot).exp()
        if kind == 1:
            theta /= f
        elif kind == 2:
            theta *= (f.ln() * (-2 * i) / (rot - 2)).exp()
        elif kind == 3:
            d = lambda x: rot * math.log(original / (2 * math.pi * x)) / (2 * math.log(base))
            a, b = max(math.floor(d(high)), 0), min(math.ceil(d(low)), rot - 1)
            g = min(max((Decimal(i) - a) / Decimal(max(b - a, 0.001)), Decimal(0)), Decimal(1))
            theta = theta * (1 - g) + theta / f * g
        elif kind == 4:
            h = min(max((n * theta / TURN - lo) / (hi - lo), Decimal(0)), Decimal(1))
            theta = theta * h + theta / f * (1 - h)
        out.append(theta / TURN)
    return out


def test_turns_are_rounded_once(turns):
    """Within 2^-65 of a turn (and a hundredth of that for the arithmetic), so that 2^31
    positions on the angle is off by 2^-34 turns."""
    getcontext().prec = 80
    r = random.Random(5)
    cases = [(4, 1.298, 0, 1.0, 1.0, 1.0, 2.0), (2, 10000.0, 0, 1.0, 1.0, 1.0, 2.0), (4, 10000.0, 2, 8.0, 1.0, 1.0, 2.0)]
    for _ in range(60):
        kind = r.randrange(5)
        cases.append((2 * r.randrange(2, 129), r.choice([10000.0, 500000.0, 1e6, 1 + r.random(), 10 ** r.uniform(0.1, 200)]),
                      kind, r.choice([1.0, 2.0, 8.0, 0.5, 32.0, r.uniform(0.01, 60)]), r.choice([4096.0, 8192.0, 1e5]),
                      r.choice([1.0, 0.7]), r.choice([4.0, 32.0])))
    for case, (ok, *got) in zip(cases, turns(cases)):
        assert ok == 1
        for t, x in zip(got, expected(*case)):
            off = abs(Decimal(t) / 2 ** 64 - x % 1)
            assert min(off, 1 - off) * 2 ** 64 <= Decimal("0.505"), case


def test_bases_and_factors_at_the_ends_of_float64(turns):
    rows = turns([(64, 1e300, 0, 1.0, 1.0, 1.0, 2.0), (64, 1.7e308, 1, 1.7e308, 1.0, 1.0, 2.0),
                  (64, 1.0000000000000002, 0, 1.0, 1.0, 1.0, 2.0), (64, 10000.0, 2, 1e300, 1.0, 1.0, 2.0)])
    first = int(Decimal(2 ** 64) / TURN + Decimal("0.5"))
    assert all(r[0] == 1 for r in rows) and rows[0][1] == rows[3][1] == first
    assert rows[1][1:] == [0] * 32 and all(abs(t - first) < 2 ** 13 for t in rows[2][1:])
    # a pair that turns more than 2^24 times a position is refused
    assert [r[0] for r in turns([(64, 10000.0, 1, 1e-9, 1.0, 1.0, 2.0), (64, 10000.0, 4, 1e-300, 64.0, 1.0, 2.0),
                                 (64, 10000.0, 1, 2.0 ** -24, 1.0, 1.0, 2.0)])] == [0, 0, 1]

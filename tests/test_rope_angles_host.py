"""The rotation's angle per position as a 64-bit fraction of a turn, against exact
arithmetic (no GPU): the function is compiled by itself."""
import math
import os
import random
import subprocess
from fractions import Fraction

import pytest

from attention_swa_forward_gb300 import build as B
from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import RopeGeometry

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_swa_forward_gb300", "csrc")
# 60 decimals of 2 pi
TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def frequencies():
    g = random.Random(5)
    fixed = [0.0, 1.0, -1.0, 1e-4, -1e-4, 1e-15, -1e-15, 1e-30, -1e-300, 5e-324, 700.25, -700.25, 2.0 ** 20, -2.0 ** 20,
             2.0 ** 20 - 2.0 ** -32, 2 * math.pi, -2 * math.pi, math.pi, 123456.789, 1048575.123456]
    drawn = [g.choice((-1, 1)) * math.exp(g.uniform(math.log(1e-12), math.log(2.0 ** 20))) for _ in range(400)]
    return fixed + drawn + [10000.0 ** (-2.0 * i / 128) for i in range(64)]


@pytest.fixture(scope="module")
def fraction_of(tmp_path_factory):
    d = tmp_path_factory.mktemp("turn")
    (d / "turn.cpp").write_text('#include <cstdio>\n#include "swa_turn.h"\nint main() {\n  double f;\n'
                                '  while (std::scanf("%lf", &f) == 1)\n'
                                '    std::printf("%llu\\n", (unsigned long long)swa::turn_fraction(f));\n}\n')
    subprocess.run(["g++", "-O3", "-std=c++17", "-I", CSRC, str(d / "turn.cpp"), "-o", str(d / "turn")], check=True)

    def call(fs):
        text = "".join(f"{f.hex()}\n" for f in fs)
        r = subprocess.run([str(d / "turn")], input=text, capture_output=True, text=True, check=True)
        return [int(x) for x in r.stdout.split()]

    return call


def test_fractions_are_the_nearest(fraction_of):
    """Within half a step of 2^-64 turns, and the 2^-20 of a step that the 64-bit
    arithmetic of the remainder may add: the product's low part, below 2^28
    steps, is rounded relatively by 2^-53 in each of its three operations."""
    fs = frequencies()
    for f, got in zip(fs, fraction_of(fs)):
        off = (got - Fraction(f) / TWO_PI * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 2 ** 20), (f, float(off))


def test_an_opposite_frequency_turns_as_far_back(fraction_of):
    fs = frequencies()
    for a, b in zip(fraction_of(fs), fraction_of([-f for f in fs])):
        assert (a + b) % 2 ** 64 == 0


@pytest.mark.parametrize("base", [math.inf, math.nan, 0.0, -1.0, 1e-320, 1e-300])
def test_a_base_without_frequencies_is_refused_from_python_too(base):
    """RopeParams forms the default frequencies; the refusal is the library's.
    (Positions off their alignment, checked after the parameters, keep any call
    from being made.)"""
    B.build()
    p = swa.RopeParams(RopeGeometry("TND", 1, 16, 4, 64, base=base))
    st = swa.lib().swa_rope_forward(p.ref(), 1 << 20, None, None, None, (1 << 20) + 2, 1 << 20, None, None, None, None)
    assert st == swa.SWA_ERR_PARAM_INVALID
    assert "base" in swa.swa_last_error() or "inv_freq" in swa.swa_last_error()

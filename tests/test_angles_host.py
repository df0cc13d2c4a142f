"""Cosine and sine of position times frequency (csrc/fa_angle.h), compiled for the
host with checks for undefined behaviour, against exact rational arithmetic: no GPU
needed."""
import math
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "io_aware_exact_35_b200", "csrc")
TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194988918")

_PROGRAM = r"""
#include "fa_angle.h"
#include <cstdio>
int main() {  // (position, frequency) in, (cos, sin) out
  struct { int pos; float f; } in;
  float out[2];
  while (std::fread(&in, sizeof in, 1, stdin) == 1) {
    fa::rope::turn(in.pos, fa::rope::turns(in.f), out[0], out[1]);
    std::fwrite(out, sizeof out, 1, stdout);
  }
}
"""


@pytest.fixture(scope="module")
def angles(tmp_path_factory):
    """(positions, frequencies) -> [n, 2] cosines and sines; undefined behaviour aborts."""
    at = tmp_path_factory.mktemp("angles")
    source, program = at / "angles.cpp", at / "angles"
    source.write_text(_PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", "-fsanitize=undefined,float-cast-overflow",
                    "-fno-sanitize-recover=all", "-fsanitize-undefined-trap-on-error", str(source), "-o",
                    str(program)], check=True, capture_output=True)

    def run(pos, freq):
        data = np.empty(len(pos), dtype=[("pos", np.int32), ("f", np.float32)])
        data["pos"], data["f"] = pos, freq
        r = subprocess.run([str(program)], input=data.tobytes(), capture_output=True)
        assert r.returncode == 0, f"stopped by signal {-r.returncode} (undefined behaviour)"
        return np.frombuffer(r.stdout, dtype=np.float32).reshape(-1, 2)
    return run


def _check(got, pos, freq):
    for (c, s), p, f in zip(got, pos, freq):
        theta = Fraction(int(p)) * Fraction(float(f))
        theta = float(theta - (theta / TWO_PI).__round__() * TWO_PI)
        # the angle carries three roundings of 2^-24 (integer to float, the factor,
        # the product) of at most pi / 4, the series about two and their remainder half of one
        for have, want in ((c, math.cos(theta)), (s, math.sin(theta))):
            assert abs(float(have) - want) <= 6 * 2.0 ** -24, (p, f, have, want)


def test_all_quarters_of_a_turn(angles):
    """Angles all around the turn, the border of the integer range among them."""
    n = 4096
    freq = np.full(n, 2 * math.pi / n, dtype=np.float32)
    pos = np.arange(n)
    _check(angles(pos, freq), pos, freq)
    _check(angles(-pos, freq), -pos, freq)


def test_far_positions(angles):
    rng = np.random.default_rng(5)
    pos = np.concatenate((rng.integers(-2 ** 31, 2 ** 31, 3000), [0, 1, -1, 2 ** 31 - 1, -2 ** 31]))
    freq = np.exp(rng.uniform(math.log(1e-7), math.log(2.0), len(pos))).astype(np.float32)
    freq[::5] *= -1
    freq[:3] = 0.0, 1.0, 2.0 ** -20
    _check(angles(pos, freq), pos, freq)


def test_frequencies_that_are_no_finite_numbers(angles):
    pos = np.array([0, 1, -7, 2 ** 31 - 1])
    for f in (math.inf, -math.inf, math.nan):
        assert np.isnan(angles(pos, np.full(4, f, dtype=np.float32))).all()


def test_least_and_largest_frequencies(angles):
    """Frequencies about the least fraction that is held (2^-64 of a turn is
    3.4e-19), denormal and very large ones."""
    tiny = np.array([3.3e-19, 3.5e-19, 5e-19, 6.7e-19, 7e-19, 1.4e-45, 1e-38], dtype=np.float32)
    freq = np.concatenate((tiny, -tiny))
    for p in (0, 1, -1, 2 ** 31 - 1, -2 ** 31):
        pos = np.full(len(freq), p)
        _check(angles(pos, freq), pos, freq)
    big = np.array([3.4e38, 1e30, 2.0 ** 60], dtype=np.float32)
    got = angles(np.array([0, 3, -5]), big)
    assert np.isfinite(got).all() and np.abs(np.hypot(*got.T) - 1).max() <= 2.0 ** -20

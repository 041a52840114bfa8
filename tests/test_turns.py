"""The rotation's frequencies in fixed point (turns.h) against decimals of 60
digits: within the stated error, for positions that fill 63 bits.  The fractions
come from a host program."""
import os
import random
import shutil
import subprocess
from decimal import Decimal, getcontext

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "head_context_attention_gb300", "csrc")
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def test_turn_fractions_within_their_bound(tmp_path):
    getcontext().prec = 60
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "turns"
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "turns.cpp"), "-o", str(exe)],
                   check=True, capture_output=True)
    rng = random.Random(1)
    freqs = [base ** (-2.0 * i / 128) for base in (10000.0, 500000.0) for i in range(64)]
    freqs += [10.0 ** rng.uniform(-18, 18) for _ in range(200)] + [6.283185307179586, 1e300, 5e-324]
    freqs += [-f for f in freqs] + [0.0]
    out = subprocess.run([str(exe)] + [f.hex() for f in freqs], check=True, capture_output=True, text=True).stdout.split()
    assert len(out) == len(freqs)
    for f, fraction in zip(freqs, map(int, out)):
        for p in (1, 131072, -(2 ** 31), 2 ** 45 + 12345, -(2 ** 55) + 1, 2 ** 63 - 1):
            turns = p * fraction % 2 ** 64
            with_ = Decimal(turns) / 2 ** 64 * TWO_PI
            # beyond 60 digits of pi an angle is not known here
            if abs(p * f) > 1e30:
                continue
            far = abs(with_ - Decimal(p) * Decimal(f) % TWO_PI) % TWO_PI
            far = min(far, TWO_PI - far)
            assert far <= abs(p) * (Decimal(abs(f)) * Decimal(2) ** -52 + TWO_PI * Decimal(2) ** -64), (f, p)

"""Sine and cosine of a 64-bit fraction of a turn (CPU): csrc/vq_turn.cuh compiled for the host, against the angle in more bits."""
import ctypes
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from bit_vector_quantized_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286209, 10 ** 78)


def exact(turn):
    """(sine, cosine) by their series in fractions, rounded once: the nearest quarter turn taken off."""
    q = (turn + (1 << 61)) >> 62
    x = 2 * PI * Fraction(turn - (q << 62), 1 << 64)
    s, c, term = Fraction(0), Fraction(0), Fraction(1)
    for n in range(26):
        if n % 2:
            s += term * (1 if n % 4 == 1 else -1)
        else:
            c += term * (1 if n % 4 == 0 else -1)
        term = Fraction(int(term * x / (n + 1) * (1 << 160)), 1 << 160)
    s, c = ((s, c), (c, -s), (-s, -c), (-c, s))[q % 4]
    return float(s), float(c)


def test_against_fractions(tmp_path):
    try:
        nvcc = build._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    lib = str(tmp_path / "turn_host.so")
    subprocess.check_call([nvcc, *build.ARCH, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-o", lib, os.path.join(HERE, "turn_host.cu")])
    rng = np.random.default_rng(1)
    turns = [int(x) for x in rng.integers(0, 2 ** 64, 3000, dtype=np.uint64)]
    for q in range(8):  # eighths of a turn and what lies around them
        turns += [(q << 61) + d & (2 ** 64 - 1) for d in (-(1 << 40), -3, -1, 0, 1, 2, 1 << 20, 1 << 50)]
    turns = np.array(turns, np.uint64)
    si, co = np.empty(len(turns)), np.empty(len(turns))
    P = ctypes.c_void_p
    fn = ctypes.CDLL(lib).turn_sincos_host
    fn.argtypes = [P, ctypes.c_longlong, P, P]
    fn(turns.ctypes.data, len(turns), si.ctypes.data, co.ctypes.data)
    want = np.array([exact(int(t)) for t in turns])
    # Of x and its product 2 2^-53 relative, the series' sums (1 ulp of the last two, x^17 / 17!): under 4 2^-53 of 1, and of a
    # sine or cosine near zero, which is x but for what x2 takes, under 4 2^-53 of itself.
    for got, w in ((si, want[:, 0]), (co, want[:, 1])):
        assert (np.abs(got - w) <= 4 * 2.0 ** -53 * np.where(np.abs(w) < 0.7, np.abs(w), 1)).all()

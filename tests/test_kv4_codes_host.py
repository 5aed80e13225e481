"""The 4-bit cache's codes at half-way points, of groups whose values differ so much in size that x - m is no fp32 or fp64
number: the oracle against rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

import oracle.kv4_oracle as KV
from synth.workloads import bf16_round


def half_way_groups(seed, n=256):
    """[n, 32] bf16 groups with step s (3 bits and a power of two), values at (k + 1/2) s above 0 or above the minimum, and
    either a minimum or other values tiny next to s, of both signs: 2^-10 to 2^-120 of it."""
    g = np.random.default_rng(seed)
    x = np.zeros((n, 32))
    for i in range(n):
        s = g.choice([1.0, 1.25, 1.5]) * 2.0 ** g.integers(-20, 20)
        tiny = s * 2.0 ** -float(g.integers(10, 120)) * (1 + g.integers(0, 128) / 128)
        if i % 2 == 0:  # a tiny minimum, and half-way points that it falls short of
            x[i] = (g.integers(0, 15, 32) + 0.5) * s
            x[i, :2] = tiny, 15 * s
        else:  # tiny values on either side of 0, which is half-way above the minimum
            k = int(g.integers(1, 14))
            x[i] = g.choice([-tiny, tiny, 0.0, tiny * 2.0 ** -5], 32)
            x[i, :2] = -(k + 0.5) * s, (14.5 - k) * s
        x[i] = g.permutation(x[i])
    return bf16_round(x.astype(np.float32))


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_the_oracles_codes_are_exact(seed):
    x = half_way_groups(seed).reshape(-1, 128)
    codes, step, low = KV.quantise(x)
    s, m = (np.repeat(KV._bf16_value(t), 32, -1) for t in (step, low))
    assert np.all(s > 0)
    short = 0
    for c, v, a, b in zip(codes.flat, x.flat, s.flat, m.flat):
        q = (Fraction(float(v)) - Fraction(float(b))) / Fraction(float(a)) + Fraction(1, 2)
        assert int(c) == q.__floor__(), (v, b, a)
        short += np.floor(float(np.float32(np.float32(v) - np.float32(b))) / float(a) + 0.5) != int(c)
    assert short > 500  # where x - m rounded to nearest in fp32 would give another code


def test_the_case_of_a_tiny_minimum():
    x = np.zeros((1, 64))
    x[0, :3], x[0, 32:35] = [2.0 ** -30, 15.0, 7.5], [-7.5, 7.5, -2.0 ** -30]
    x[0, 3:32] = 1.0
    codes, step, _ = KV.quantise(x)
    assert KV._bf16_value(step).tolist() == [[1.0, 1.0]]
    assert codes[0, :3].tolist() == [0, 15, 7] and codes[0, 32:36].tolist() == [0, 15, 7, 8]

"""The angles of the rotary positions, to units of their sines and cosines themselves, and frequencies that are no numbers.

The reference's angle is exact: positions and frequencies are integers and binary fractions, and the fraction of a turn
is formed in integers with 200 bits of pi.

Units of 2^-24.  The fraction of a turn is good to 2^-64 of a turn per position; with a remainder of r turns off the
nearest quarter, rounded once to FP32 (half a unit of r), sincospif is good to 2 ulp (2 units of a value in [1/2, 1], 4 of
one just above a power of two): sin and cos of the remainder are within 5 units of themselves.  A quarter turn only swaps
them.  The rotation of (1, 0) is a product by 1 and one by 0.
"""
import math

import numpy as np
import pytest
import torch

from gate_cores_b200 import cores

from .close64 import f64, same_bits
from .test_gpu_rope import DT, qk

pytestmark = pytest.mark.gpu

BITS = 200


def _pi():
    """pi in units of 2^-(BITS + 64): 16 atan(1/5) - 4 atan(1/239)."""
    one = 1 << (BITS + 64)

    def atan_inv(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    return 4 * (4 * atan_inv(5) - atan_inv(239))


PI = _pi()


def turn_of(freq, pos):
    """pos * freq modulo 2 pi in (-pi, pi], as a float good to 2^-53 of itself."""
    num, den = float(freq).as_integer_ratio()
    phi = (num * pos << (BITS + 64)) // den  # in units of 2^-(BITS + 64), exact where freq has few bits below 2^-200
    phi %= 2 * PI
    if phi > PI:
        phi -= 2 * PI
    return phi / (1 << (BITS + 64))


def unit_vectors(freqs, positions, backward=False):
    """(cos, sin) of each position (a row) and frequency, from the rotation of (1, 0)."""
    n = len(freqs)
    q = torch.zeros(len(positions), 1, 2 * n)
    q[..., :n] = 1.0
    f = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    pos = torch.tensor(positions, dtype=torch.int64).to(torch.int32).cuda()
    call = cores.rope_backward if backward else cores.rope
    y = call(q.cuda(), None, f, positions=pos, pairing="half")[0][:, 0]
    return y[:, :n], y[:, n:]


# slow pairs (a millionth of a turn per position and less), ordinary ones, and ones of many turns per position
FREQS = [1e-9, 2.3e-8, 1.4e-7, 1.3e-6, 7.7e-5, 0.01, 1.0, -0.3, 3.0, 100.0, -1234.5, 2.0 ** 20 + 0.375, 1.7 * 2 ** 33, 1.1 * 2 ** 42,
         5e-324, 0.0]
POSITIONS = [0, 1, -1, 2, 3, 17, 1000, 65535, 131071, -131072, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31]


def test_sines_are_good_to_units_of_themselves(cuda_ok):
    c, s = (f64(t) for t in unit_vectors(FREQS, POSITIONS))
    for i, p in enumerate(POSITIONS):
        for j, f in enumerate(FREQS):
            phi = turn_of(f, p)
            # the fraction itself: half a unit of 2^-64 turns for each of its two parts, times the position, and (pairs of
            # many turns) what 1 / 2 pi in two doubles leaves, 2^-107 of the turns
            turns = abs(p) * (2.0 ** -64 + abs(f) * 2.0 ** -107)
            slack = 2 * math.pi * turns
            for got, want in ((c[i, j], math.cos(phi)), (s[i, j], math.sin(phi))):
                assert abs(got - want) <= 5 * 2.0 ** -24 * abs(want) + slack, (p, f, got, want)


def test_turning_back_is_turning_by_the_negative_position(cuda_ok):
    pos = [p for p in POSITIONS if p != -2 ** 31]
    fwd, back = unit_vectors(FREQS, [-p for p in pos]), unit_vectors(FREQS, pos, backward=True)
    assert torch.equal(fwd[0], back[0]) and torch.equal(fwd[1], back[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("pairing,rd", [("interleaved", 20), ("half", 16), ("half", 20)])
def test_a_frequency_that_is_no_number(cuda_ok, bad, dt, pairing, rd):
    # the formula's cos and sin are NaN at every position, and so are the pair's elements; the other pairs are as before
    q, k = qk(9, 3, 1, 64, DT[dt])
    pos = torch.tensor([0, 1, 2, -5, 77, 131071, 9, 10, 2 ** 31 - 1], dtype=torch.int32).cuda()
    f = cores.rope_frequencies(rd)
    wrong = f.clone()
    wrong[3] = bad
    pair = [3, 3 + rd // 2] if pairing == "half" else [6, 7]
    others = [i for i in range(64) if i not in pair]
    for call in (cores.rope, cores.rope_backward):
        want, got = call(q, k, f, positions=pos, pairing=pairing), call(q, k, wrong, positions=pos, pairing=pairing)
        for w, g in zip(want, got):
            assert torch.isnan(g[..., pair]).all()
            assert same_bits(g[..., others], w[..., others])


@pytest.mark.parametrize("far", [1e17, -3e25, 1e300, -1.7e308])
def test_a_finite_frequency_however_large_is_a_rotation(cuda_ok, far):
    # beyond 2^43 the angle is less and less exact, but it stays an angle
    c, s = (f64(t) for t in unit_vectors([far, 0.5], [1, 3, -7, 2 ** 31 - 1]))
    # each of the two within 5 units of itself, twice in its square
    assert np.all(np.abs(c * c + s * s - 1) <= 2 * 5 * 2.0 ** -24 * 1.01)
    assert np.all(np.abs(c[:, 1] - np.cos([math.fmod(0.5 * p, 2 * math.pi) for p in (1, 3, -7, 2 ** 31 - 1)])) < 1e-5)

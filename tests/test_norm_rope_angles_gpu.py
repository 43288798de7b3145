"""The rotation's angles at far positions and high frequencies, on the GPU
against integers: position * inv_freq / 2 pi modulo a turn from 100 digits of pi.

The header's bound is 2^-25 turns plus |position| (2^-62 + 2^-106 |inv_freq|).
Pairs (1, 0) turn to (cos t, sin t): the angle's error, and 8 u (u = 2^-24) for
the sine, the cosine and their product with 1."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _two_pi():
    one = 10 ** 100

    def arctan_inverse(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    return Fraction(8 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)  # Machin's formula


FREQUENCIES = [1.0, 1e-6, 0.1, 3.0, 10.0, -10.0, 100.0, 1000.0, 12345.678, -0.3, 1e6, 1e9, -1e12, 2.0 ** 40, 1e-30, 0.0]
POSITIONS = [0, 1, -1, 2, 65535, 1_000_003, -1_000_003, 2 ** 31 + 7, 2 ** 40 + 12345, -(2 ** 40) - 3, 2 ** 45 + 1]


def test_angles_at_far_positions_and_high_frequencies(uly):
    two_pi = _two_pi()
    n, d = len(POSITIONS), 64
    x = torch.zeros(1, 1, n, 1, d, device="cuda")
    x[..., 0:32:2] = 1.0  # interleaved pairs (1, 0)
    y = [torch.empty_like(x) for _ in range(2)]
    pos = torch.tensor(POSITIONS, device="cuda").view(1, 1, n)
    uly.ulysses_qkv_norm_rope_fwd(x, x.clone(), None, *y, None, 1, inv_freq=np.array(FREQUENCIES), positions=pos,
                                  interleaved=True)
    got = y[0][0, 0, :, 0].cpu().double().numpy()
    for i, p in enumerate(POSITIONS):
        for f, w in enumerate(FREQUENCIES):
            turns = Fraction(w) * p / two_pi
            t = 2 * math.pi * float(turns - math.floor(turns))
            tol = 2 * math.pi * (2.0 ** -25 + abs(p) * (2.0 ** -62 + abs(w) * 2.0 ** -106)) + 8 * 2.0 ** -24
            c, s = got[i, 2 * f], got[i, 2 * f + 1]
            assert abs(c - math.cos(t)) <= tol and abs(s - math.sin(t)) <= tol, (p, w, c, s, t)

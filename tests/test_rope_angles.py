"""Angles of duo_qk_norm_rope over the whole accepted range of frequencies (0 to 10^6
radians per position) and positions (any int32), against exact arithmetic: the angle in
turns as a fraction of integers.

Rows of ones and zeros turn (1, 0) into (cos, sin), without another rounding at fp32.
Tolerance: sincospif's two units of the last place, 2^-22; its argument, a number of half
turns below one, rounded to fp32 and, before that, cut off at 2^-32 turns: pi 2^-24 +
2 pi 2^-32.  In all 4.3e-7."""
import math
import random
from fractions import Fraction

import pytest
import torch

from head_split_kv_duo_b200.duo import DuoRope

DEV = "cuda"
TOL = 2.0 ** -22 + math.pi * 2.0 ** -24 + 2 * math.pi * 2.0 ** -32


def pi_fraction(bits=400):
    """pi by Machin's formula, 16 arctan(1/5) - 4 arctan(1/239), below 2^-bits off."""
    one = 1 << (bits + 20)

    def arctan_inverse(x):
        total, power, k = 0, one // x, 0
        while power:
            total += (-1) ** k * (power // (2 * k + 1))
            power //= x * x
            k += 1
        return total
    return Fraction(16 * arctan_inverse(5) - 4 * arctan_inverse(239), one)


TURN = 2 * pi_fraction()


def cos_sin(position, inv_freq):
    turns = position * Fraction(inv_freq) / TURN
    a = 2 * math.pi * float(turns - round(turns))
    return math.cos(a), math.sin(a)


def test_pi():
    assert float(TURN) == 2 * math.pi and abs(TURN - 2 * Fraction(math.pi)) < Fraction(1, 1 << 50)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_are_exact_for_any_position_and_frequency(interleaved):
    r = random.Random(3)
    f = [0.0, 5e-324, 1e-310, 1e-30, 2.0 ** -40, 1e-7, 0.1, 1.0, 6.2, 2 * math.pi, 6.4, 100.0, 12345.678, 2.0 ** 17,
         999999.9, 1e6, 978234.1742832669, 985576.6942154213]
    f += [math.exp(r.uniform(math.log(1e-6), math.log(1e6))) for _ in range(24)]
    f += [r.uniform(5e5, 1e6) for _ in range(64 - len(f))]
    pos = [0, 1, -1, 2, 1 << 20, 2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 2] + \
        [r.randrange(-(2 ** 31), 2 ** 31) for _ in range(56)]
    x = torch.zeros(len(pos), 1, 128, device=DEV)
    first = torch.arange(64, device=DEV) * (2 if interleaved else 1)
    second = first + (1 if interleaved else 64)
    x[..., first] = 1
    out, _, _ = DuoRope(128, f, interleaved=interleaved).norm_rope(
        x, None, torch.tensor(pos, dtype=torch.int32, device=DEV))
    want = torch.tensor([[cos_sin(p, g) for g in f] for p in pos], dtype=torch.float64)  # [n][64][2]
    got = torch.stack((out[:, 0, first], out[:, 0, second]), -1).double().cpu()
    off = (got - want).abs().amax(-1)
    worst = divmod(int(off.argmax()), 64)
    assert off.max() <= TOL, f"off by {float(off.max())} at position {pos[worst[0]]}, inv_freq {f[worst[1]]}"

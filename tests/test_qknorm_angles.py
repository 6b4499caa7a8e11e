"""Rotations by large angles.  The reference reduces position x frequency in whole numbers with 400 bits of pi.
A frequency over 2 pi is rounded to 2^-65 of a turn, 2^-34 times 2^31 positions; the angle enters the sine as 32
bits of a turn (2^-32) rounded to 24 bits (2^-25 of half a turn at most: 2^-23 radians); sine and cosine are within
2 steps of 2^-24 of themselves and the products with 1 and 0 are exact: 2^-21 covers all."""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu


def two_pi(bits=400):
    """floor(2 pi 2^bits): pi = 16 atan(1/5) - 4 atan(1/239)."""
    def atan(n):
        total, term, k = 0, (1 << bits + 32) // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    return 2 * (16 * atan(5) - 4 * atan(239)) >> 32


TWO_PI = Fraction(two_pi(), 1 << 400)


def angle(position, freq):
    turn = Fraction(position) * Fraction(freq) / TWO_PI
    turn -= math.floor(turn)
    return 2 * math.pi * float(turn if turn < Fraction(1, 2) else turn - 1)


FREQS = [1.0, 100.25, 1000.123, 12345.678, 65536.0, 99999.999, 2.0 ** 20, 2.0 ** 20 - 2.0 ** -32, -1048575.77, 2 * math.pi,
         -2 * math.pi * 1e5, math.pi, 1e-3, 1e-12, 2.0 ** -33, 2.0 ** -63, 3e-20, 1e-300, 5e-324, 0.0, -0.0, 0.5, 3.0, 7e5]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("pad", [0, 1])
def test_large_angles(kda, inter, pad):
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 123456789, -987654321, 131072, 1, -1, 0]
    half = len(FREQS)
    heads = torch.zeros(len(pos), 1, 2 * half + 8 * (half % 4))
    a = slice(0, 2 * half, 2) if inter else slice(0, half)
    b = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
    heads[..., a] = 1.0
    wide = torch.zeros(len(pos), heads.shape[-1] + 4 + pad).cuda()  # pad 1: single channels at a time
    q = wide[:, pad:pad + heads.shape[-1]].unflatten(-1, (1, -1))
    q.copy_(heads)
    y, _ = kda.qknorm_fwd(q, None, torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(FREQS, dtype=torch.float64).cuda(),
                          interleaved=inter)
    back, *_ = kda.qknorm_bwd(q, None, y, None, torch.tensor(pos, dtype=torch.int32).cuda(),
                              torch.tensor(FREQS, dtype=torch.float64).cuda(), interleaved=inter)
    y = y.cpu().double()
    for i, p in enumerate(pos):
        for j, f in enumerate(FREQS):
            x = angle(p, f)
            assert abs(y[i, 0, a][j] - math.cos(x)) <= 2.0 ** -21, (p, f)
            assert abs(y[i, 0, b][j] - math.sin(x)) <= 2.0 ** -21, (p, f)
    assert ((back.cpu() - heads).abs() <= 2.0 ** -20).all()

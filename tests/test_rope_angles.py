"""Angles of rotary positions against exact ones: how far they may be off, at the ends
of positions and for frequencies of more than a turn."""
import math
from fractions import Fraction

import pytest
import torch

import exact_attention_58_gb300 as ea

FREQS = [1.0, 0.5, 1e-3, 1e-8, -0.3, 3.1415927, 6.2831855, 7.5, -12.0, 1000.25, 54321.0, -1e6, 0.99999994, 2.0**-40, 0.0, 1.5e7]
POSITIONS = [0, 1, -1, 2, 999, 12345, -70001, 2**24 + 1, 2**30 - 1, 2**31 - 1, -2**31]


def _atan_inverse(n, bits):
    """arctan(1 / n) times 2^bits."""
    total, term, k = 0, (1 << bits) // n, 1
    while term:
        total += term // k if k % 4 == 1 else -(term // k)
        term //= n * n
        k += 2
    return total


# pi = 16 arctan(1/5) - 4 arctan(1/239) (Machin), 200 bits
PI = Fraction(16 * _atan_inverse(5, 220) - 4 * _atan_inverse(239, 220), 1 << 220)


def exact_turns(t, f):
    """t f / (2 pi) of the float32 f, in [0, 1)."""
    x = t * Fraction(f) / (2 * PI)
    return x - math.floor(x)


def bound(t, f):
    return abs(t) * max(1.0, abs(f)) * 2.0**-53 + 2.0**-25


def test_pi():
    assert float(PI) == math.pi and abs(exact_turns(1, 2 * math.pi) - Fraction(1, 1)) < Fraction(1, 10**15)


def kernel_turns(t, f):
    """The kernel's steps, in Python: the fraction of a turn per position to 64 bits, their
    product modulo 2^64, its upper 32 bits."""
    turns = f * 0.15915494309189533577
    step = min(int((turns - math.floor(turns)) * 2.0**64), 2**64 - 1)
    return Fraction((t * step % 2**64) >> 32, 1 << 32)


@pytest.mark.parametrize("t", POSITIONS)
def test_steps_are_within_the_bound(t):
    for f in torch.tensor(FREQS).tolist():
        d = kernel_turns(t, f) - exact_turns(t, f)
        d = abs(d - round(d))
        assert d <= bound(t, f), (t, f, float(d))


def test_the_frequency_counts():
    """Above a turn the error grows with the frequency: without that factor it is too little."""
    t, f = 2**31 - 1, 1000.25
    d = kernel_turns(t, f) - exact_turns(t, f)
    assert abs(d - round(d)) > abs(t) * 2.0**-53 + 2.0**-25


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_cosines_and_sines(dtype, interleaved):
    """Pairs (1, 0): the result is the cosine and the sine."""
    f = torch.tensor(FREQS)
    pos = torch.tensor(POSITIONS, dtype=torch.int32)
    x = torch.zeros(len(POSITIONS), 1, 64, dtype=dtype)
    first, second = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    x[..., first] = 1.0
    y = ea.attn_rope(x.cuda(), None, f.cuda(), pos.cuda(), interleaved=interleaved)[0].double().cpu()
    fast = 2.0**-22 if dtype is torch.float32 else 2.0**-20
    for i, t in enumerate(POSITIONS):
        for k, w in enumerate(f.tolist()):
            turn = 2 * math.pi * float(exact_turns(t, w))
            # the angle's, the function's, and the result's rounding
            tol = 2 * math.pi * bound(t, w) + fast + torch.finfo(dtype).eps / 2
            assert abs(float(y[i, 0, first][k]) - math.cos(turn)) <= tol, (t, w)
            assert abs(float(y[i, 0, second][k]) - math.sin(turn)) <= tol, (t, w)

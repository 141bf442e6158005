"""Sines and cosines of the rotary embedding to the last bits of fp32, at any position and frequency."""
import math
from fractions import Fraction

import pytest
import torch

import cluster_routed_sparse_b200 as crs

pytestmark = pytest.mark.gpu

# 2 pi to 60 digits (from its decimal expansion)
TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194988918")


def turned(pos, freqs):
    """(cos, sin) of every position and frequency, as the kernel forms them in fp32: (1, 0) rotated."""
    x = torch.zeros(1, 1, len(pos), 2 * len(freqs), device="cuda")
    x[..., 0::2] = 1
    p = torch.tensor(pos, device="cuda", dtype=torch.int32).view(-1, 1)
    y = crs.rope_axes(x, None, p, (len(freqs),), freqs=freqs)[0, 0].double().cpu()
    return y[:, 0::2], y[:, 1::2]


def exact(pos, freqs):
    c, s = torch.zeros(2, len(pos), len(freqs), dtype=torch.float64)
    for i, p in enumerate(pos):
        for j, f in enumerate(freqs):
            turn = (p * Fraction(f) / TWO_PI) % 1
            turn = turn - 1 if turn > Fraction(1, 2) else turn
            c[i, j], s[i, j] = math.cos(2 * math.pi * float(turn)), math.sin(2 * math.pi * float(turn))
    return c, s


def close(pos, freqs):
    # the angle: 2^-32 turns, pi 2^-31 rad; sine and cosine of a float: 1 ulp, 2^-23 relative; the bits of the angle
    # that a float does not hold, pi 2^-24 at most, come in by a product and a sum: half an ulp, and half their square
    angle = math.pi * 2.0 ** -31 + (math.pi * 2.0 ** -24) ** 2 / 2
    for got, want in zip(turned(pos, freqs), exact(pos, freqs)):
        tol = 1.5 * 2.0 ** -23 * want.abs() + angle
        assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())


def test_small_sines():
    """Angles near half a turn and a whole one, where sines are small."""
    near = [math.pi * (n + e) for n in (1, 2, -1, 0.5) for e in (1e-3, -1e-3, 3e-5, 0.01, -0.003, 0.1)]
    close([1, -1, 3, 1001], [float(f) for f in near if abs(f) < 2 * math.pi])


def test_random_angles():
    g = torch.Generator().manual_seed(1)
    f = (torch.rand(128, generator=g, dtype=torch.float64) * 6).tolist()
    close([0, 1, 7, 4095, 75599, 10 ** 6 + 3, 2 ** 31 - 1, -2 ** 31], f)


def test_frequencies_above_a_turn():
    """More than one turn a step: whole turns leave, the fraction keeps all its bits."""
    close([1, 13, 75599, 2 ** 31 - 1, -2 ** 31], [6.5, 50.0, 1000.3, -12345.678, 1e6, 2.0 ** 40 + 0.25, -1e12 / 3, 2.0 ** 52 + 1])

"""The phase of far positions: position * frequency modulo a turn, for positions
up to 2^53 and frequencies that are no fraction of a turn, against exact
rational arithmetic with pi to 400 bits.

Tolerance of the rotation: at the farthest positions the turns, within 5/8, are
rounded to fp32 by at most 2^-25, which is an angle of pi 2^-24; sine and cosine
are off by 2 units of 2^-24 more, the products and the sum by 3 half steps: under
2^-21 (|a| + |b|), then half a step of the type of the result."""
import math
import random
from fractions import Fraction

import pytest
import torch

BITS = 400
POSITIONS = [0, 1, -1, (1 << 20) + 7, -(1 << 30) - 3, (1 << 36) + 12345, (1 << 40) + 1, -(1 << 44) - 99,
             (1 << 47) + 5, (1 << 50) - 27, -(1 << 52) - 1, (1 << 53) - 1, 1 - (1 << 53)]


def arctan_of_inverse(n):
    """2^BITS arctan(1 / n), by its series in whole numbers."""
    t = (1 << BITS) // n
    s, k, sign = t, 1, -1
    while t:
        t //= n * n
        k += 2
        s += sign * (t // k)
        sign = -sign
    return s


TWO_PI = Fraction(8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), 1 << BITS)   # Machin


def turns(position, f):
    """position * f / (2 pi) less its nearest whole number, exactly (to 400 bits)."""
    t = Fraction(position) * Fraction(f) / TWO_PI
    return t - round(t)


def fma(a, b, c):
    return float(Fraction(a) * Fraction(b) + Fraction(c))


def in_64_bits(position, f):
    """The kernel's steps."""
    inv, rest = float.fromhex("0x1.45f306dc9c883p-3"), float.fromhex("-0x1.6b01ec5417056p-57")
    x, g = float(position), f * inv
    gl = fma(f, rest, fma(f, inv, -g))
    return fma(x, gl, fma(x, g, -float(round(x * g))))


def frequencies():
    return [10000.0 ** (-2 * i / 128) for i in range(64)]


def test_the_steps_in_64_bits_keep_the_phase():
    inv, rest = float.fromhex("0x1.45f306dc9c883p-3"), float.fromhex("-0x1.6b01ec5417056p-57")
    assert float(1 / TWO_PI) == inv and float(1 / TWO_PI - Fraction(inv)) == rest
    rng = random.Random(1)
    more = [rng.randrange(-(1 << b), 1 << b) for b in range(1, 54) for _ in range(4)]
    worst, plain = Fraction(0), {}
    for p in POSITIONS + more:
        for f in frequencies()[::3]:
            r = in_64_bits(p, f)
            d = Fraction(r) - turns(p, f)
            worst = max(worst, abs(d - round(d)))
            assert abs(r) <= (5 / 8 if abs(p) > 1 << 48 else 0.5 + 2.0 ** -6)
            t = float(p) * (f * inv)                      # without what the products round off
            d = Fraction(t - round(t)) - turns(p, f)
            b = abs(p).bit_length()
            plain[b] = max(plain.get(b, 0), abs(d - round(d)))
    assert worst <= Fraction(1, 1 << 52)
    assert plain[31] > Fraction(1, 1 << 28) and plain[53] > Fraction(1, 10)


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("norm", [False, True], ids=["rope", "norm"])
def test_rotation_at_far_positions(inter, norm):
    from gather_matmul_b200 import ops
    f, T, F16 = frequencies(), len(POSITIONS), torch.float16
    x = torch.randn(T, 256, generator=torch.Generator(device="cuda").manual_seed(71), device="cuda").to(F16)
    pos = torch.tensor(POSITIONS, device="cuda")
    freq = torch.tensor(f, dtype=torch.float64, device="cuda")
    y = torch.empty_like(x)
    if norm:                                              # the second slice has no norm
        ops.norm_rope(x, [torch.ones(128, dtype=F16, device="cuda"), None], y, [1, 1], 128, pos, freq,
                      interleaved=inter)
    else:
        ops.rope(x, y, [2], 128, pos, freq, interleaved=inter)
    angle = torch.tensor([[2 * math.pi * float(turns(p, v)) for v in f] for p in POSITIONS], dtype=torch.float64)
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    v, rel = x.cpu().double().view(T, 2, 128), torch.zeros(2, 1, dtype=torch.float64)
    if norm:
        v[:, 0] = v[:, 0] / torch.sqrt(v[:, 0].square().mean(-1, keepdim=True) + 1e-6)
        rel[0] = (128 + 8) * 2.0 ** -24
    got = y.cpu().double().view(T, 2, 128)
    if inter:
        a, b, ga, gb = v[..., 0::2], v[..., 1::2], got[..., 0::2], got[..., 1::2]
    else:
        a, b, ga, gb = v[..., :64], v[..., 64:], got[..., :64], got[..., 64:]
    mag = (2.0 ** -21 + rel) * (a.abs() + b.abs()) + 2.0 ** -25
    for g, want in ((ga, a * c - b * s), (gb, b * c + a * s)):
        assert ((g - want).abs() <= mag + 2.0 ** -11 * 1.001 * want.abs()).all()

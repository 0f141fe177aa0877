"""The rotation's angle at any 32-bit position and any frequency of the contract, of
either sign, against integers: a frequency is m 2^e exactly, 1 / (2 pi) a 256-bit
fraction from Machin's formula, and a position times both is taken modulo a turn."""
import math

import numpy as np
import pytest
import torch

import dynamic_sparse_attention_bra_b200 as bra

BITS = 256


def one_over_two_pi() -> int:
    """floor of 2^256 / (2 pi), by pi = 16 atan(1/5) - 4 atan(1/239) with 64 bits to spare."""
    one = 1 << (BITS + 64)

    def atan_inverse(n):
        total = term = one // n
        k = 1
        while term:
            term //= n * n
            k += 2
            total += -(term // k) if k % 4 == 3 else term // k
        return total
    pi = 16 * atan_inverse(5) - 4 * atan_inverse(239)
    return (one << BITS) // (2 * pi)


def turn_fraction(position: int, frequency: float) -> float:
    """position * frequency radians as a signed fraction of a turn, -1/2 .. 1/2."""
    m, e = math.frexp(frequency)
    m, e = int(m * 2 ** 24), e - 24  # an fp32 value: m 2^e
    x = position * m * one_over_two_pi()
    x = (x << e if e >= 0 else x >> -e) % (1 << BITS)
    if x >> (BITS - 1):
        x -= 1 << BITS
    return x / (1 << BITS)


def frequencies(n):
    """fp32 values of both signs, from far below 1 to the end of the contract."""
    r = np.random.default_rng(7)
    f = np.concatenate([2.0 ** r.uniform(-40, 0, n - 40), 2.0 ** r.uniform(0, 49.9, 30),
                        [1.0, 0.5, 0.01, 2.0 ** -20, 1e-30, 1e-42, 3.0, 6.2831855, 2.0 ** 49, 2.0 ** -31]])
    return np.where(np.arange(n) % 2 == 0, -f, f).astype(np.float32)


def test_the_constant_and_the_reference():
    assert one_over_two_pi() / 2 ** BITS == pytest.approx(1 / (2 * math.pi), rel=1e-15)
    for p, f in ((1, 1.0), (-3, 0.25), (1000, -0.125), (7, 2.0 ** -20)):
        t = p * f / (2 * math.pi)
        assert turn_fraction(p, f) == pytest.approx(t - round(t), abs=1e-13)


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True], ids=["forward", "inverse"])
@pytest.mark.parametrize("layout", ["halves", "interleaved", "odd_halves"])
def test_angles_of_far_positions(layout, inverse):
    """Pairs (1, 0) become (cos, sin).  Bound: the angle within 2^-31 of a turn; its fp32 value,
    2^-25 of half a turn; sine and cosine of the reduced angle, one unit in the last place of values
    up to 1 (2^-23, at 1 itself); the products with 1 and 0 are exact."""
    P = 255 if layout == "odd_halves" else 256
    f = frequencies(P)
    at = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, -2 ** 30 - 77, 1999999999, -1234567891, 100003]
    pos = torch.tensor(at, dtype=torch.int32, device="cuda")[None, :, None].expand(1, -1, 3).contiguous()
    x = torch.zeros((1, len(at), 512), device="cuda")
    one, two = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if layout == "interleaved" else (slice(0, P), slice(P, 2 * P))
    x[..., one] = 1
    s = bra.rotary_shape_for(x, None, 1, 0, (100, 100, P - 200), pos=pos, interleaved=layout == "interleaved",
                             inverse=inverse)
    y = torch.empty_like(x)
    bra.bra_rotary(s, x, None, pos, torch.from_numpy(f).cuda(), y, None)
    turns = np.array([[turn_fraction(p, float(w)) for w in f] for p in at]) * (-1 if inverse else 1)
    bound = 2 * math.pi * 2.0 ** -31 + math.pi * 2.0 ** -25 + 2.0 ** -23
    for part, want in ((one, np.cos(2 * np.pi * turns)), (two, np.sin(2 * np.pi * turns))):
        err = np.abs(y[0, :, part].double().cpu().numpy() - want)
        worst = np.unravel_index(err.argmax(), err.shape)
        assert err.max() <= bound, (err.max(), at[worst[0]], f[worst[1]])

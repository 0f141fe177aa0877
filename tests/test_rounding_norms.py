"""The norms of rounding_norms.py against the kernels' arithmetic in 64 bits with their
roundings alone: the arithmetic stays below them, and planted losses of accuracy (fewer
bits of P or dS, D left as <dO, O> of the rounded O) do not."""
import pytest
import torch

import block_reference as ref
from rounding_norms import error_norms, limits

BF = torch.bfloat16


def to_bits(x, bits):
    """x rounded to nearest with ``bits`` significant bits."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2.0 ** bits), e - bits)


def arithmetic(q, k, v, g, p_bits=8, ds_bits=8, correct=True):
    """One head's o, dq, dk, dv as the kernels form them, the fp32 steps in 64 bits."""
    q, k, v, g = (x[0].double() for x in (q, k, v, g))
    scale = q.shape[-1] ** -0.5
    s = q @ k.T * scale
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    o = (to_bits(e, p_bits) @ v / e.sum(-1, keepdim=True)).to(BF).double()
    p, dp = e / e.sum(-1, keepdim=True), g @ v.T
    d0 = (g * o).sum(-1, keepdim=True)
    ds = to_bits(p * (dp - d0), ds_bits)
    rest = ds.sum(-1, keepdim=True) if correct else torch.zeros_like(d0)
    dq = (ds @ k - rest * (to_bits(p, 8) @ k)) * scale
    dk = to_bits(p * (dp - d0 - rest), ds_bits).T @ q * scale
    dv = to_bits(p, p_bits).T @ g
    return {x: t.to(BF).double()[None] for x, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv))}


def worst(means, Lq, Lk, d, **how):
    """Each result's error norm over its limit, for K and V with the given means."""
    gen = torch.Generator().manual_seed(Lq + Lk)
    q, k, v, g = ((torch.randn((1, n, d), generator=gen) + mean).to(BF)
                  for n, mean in ((Lq, 0.0), (Lk, means[0]), (Lk, means[1]), (Lq, 0.0)))
    ok = ref.valid_states(1, Lk)
    r = ref.cross(q, k, v, 1, 1, ok, None, g)
    most = limits(error_norms(q, k, v, 1, 1, ok, r, g), r)
    return {x: float((t - r[x]).norm()) / most[x] for x, t in arithmetic(q, k, v, g, **how).items()}


SIZES = [(257, 333, 32), (200, 1025, 64), (150, 2100, 128), (64, 4097, 64)]
MEANS = [(0.0, 0.0), (0.5, 1.0)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("means", MEANS, ids=["centred", "offset"])
def test_the_arithmetic_stays_below(means, size):
    w = worst(means, *size)
    assert all(0.3 < x < 1.0 for x in w.values()), w


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_planted_losses_do_not(size):
    p = worst(MEANS[0], *size, p_bits=6)
    assert p["o"] > 1.0 and p["dv"] > 1.0, p
    s = worst(MEANS[0], *size, ds_bits=6)
    assert s["dq"] > 1.0 and s["dk"] > 1.0, s
    d = worst(MEANS[1], *size, correct=False)
    assert d["dq"] > 1.0, d

"""The 64-bit references of the conditioned block's operators: gradients
against differences, closed forms, published generator values."""
import math

import pytest
import torch

import block_reference as ref


def _cross_case(seed, B, Lq, Lk, heads, kv, d):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    return r(B, Lq, heads * d), r(B, Lk, kv * d), r(B, Lk, kv * d), r(B, Lq, heads * d)


@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 2), (3, 1)])
def test_cross_gradients_match_differences(heads, kv):
    q, k, v, g = _cross_case(0, 2, 3, 5, heads, kv, 4)
    ok = torch.tensor([[1, 1, 0, 1, 1], [1, 0, 0, 0, 0]]).bool()
    r = ref.cross(q, k, v, heads, kv, ok, grad=g)
    f = lambda q, k, v: float((ref.cross(q, k, v, heads, kv, ok)["o"] * g).sum())
    h = 1e-6
    gen = torch.Generator().manual_seed(1)
    for i, name in enumerate(("dq", "dk", "dv")):
        for _ in range(6):
            at = [torch.randint(0, n, (1,), generator=gen).item() for n in (q, k, v)[i].shape]
            x = [t.clone() for t in (q, k, v)]
            x[i][tuple(at)] += h
            up = f(*x)
            x[i][tuple(at)] -= 2 * h
            assert abs((up - f(*x)) / (2 * h) - float(r[name][tuple(at)])) < 1e-7


def test_cross_closed_forms():
    q, k, v, g = _cross_case(2, 2, 4, 6, 2, 2, 8)
    one = torch.zeros(2, 6).bool()
    one[:, 3] = True
    r = ref.cross(q, k, v, 2, 2, one, grad=g)
    assert torch.allclose(r["o"], v[:, 3:4].expand(-1, 4, -1))  # one state: its value
    assert float(r["dq"].abs().max()) < 1e-14 and float(r["dk"].abs().max()) < 1e-14
    none = ref.cross(q, k, v, 2, 2, one & False, grad=g)
    assert float(none["o"].abs().max()) == 0 and bool((none["lse"] == -math.inf).all())
    assert all(float(none[x].abs().max()) == 0 for x in ("dq", "dk", "dv"))
    alike = ref.cross(q * 0, k, v, 2, 2, one | True)  # equal scores: the mean, and log n
    assert torch.allclose(alike["o"], v.mean(1, keepdim=True).expand(-1, 4, -1))
    assert torch.allclose(alike["lse"], torch.full_like(alike["lse"], math.log(6)))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_rotation_and_relative(interleaved):
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn((1, 1, 16), generator=g, dtype=torch.float64) for _ in range(2))
    f, pairs = torch.tensor([1.0, 0.3, 0.7, 0.01, 0.2]), (1, 2, 2)
    P = lambda t, y, x: torch.tensor([[[t, y, x]]])
    turn = lambda z, p, inv=False: ref.rotary(z, 1, pairs, f, p, interleaved, inv)
    a, b = turn(q, P(5, 7, 2)), turn(k, P(3, 1, 9))
    c, d = turn(q, P(15, 17, 12)), turn(k, P(13, 11, 19))
    assert torch.allclose((a * b).sum(), (c * d).sum())  # only differences of positions count
    assert torch.allclose(turn(a, P(5, 7, 2), True), q)
    assert torch.allclose(a.norm(), q.norm())
    assert torch.equal(a[..., 10:], q[..., 10:])  # the channels past the pairs
    one = turn(q, P(1, 0, 0))
    i = (0, 1) if interleaved else (0, 5)
    assert math.isclose(float(one[0, 0, i[0]]),
                        float(q[0, 0, i[0]]) * math.cos(1) - float(q[0, 0, i[1]]) * math.sin(1))


def test_grid_positions_are_row_major():
    p = ref.grid_positions(2, 3, 4)[0]
    assert p[0].tolist() == [0, 0, 0] and p[5].tolist() == [0, 1, 1] and p[12].tolist() == [1, 0, 0]


def test_philox_published_values():
    assert ref.philox4x32(0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox4x32(2 ** 64 - 1, 2 ** 128 - 1) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_keeps_count_and_units():
    k = ref.keeps(20000, 1, 0.25, 7, 123)
    assert abs(float(k.double().mean()) - 0.75) < 5 * math.sqrt(0.25 * 0.75 / 20000)
    assert bool(ref.keeps(64, 1, 0.0, 1, 2).all()) and not bool(ref.keeps(64, 1, 1.0, 1, 2).any())
    u = ref.keeps(1000, 24, 0.5, 5, 9)
    assert all(len(set(u[i:i + 24].tolist())) == 1 for i in range(0, 1000, 24))

"""Rotary positions and dropout with the residual's sum against their 64-bit definitions."""
import math

import pytest
import torch

import block_reference as ref
import dynamic_sparse_attention_bra_b200 as bra
from test_gpu_cross import T, guarded, tokens

pytestmark = pytest.mark.gpu


def freqs(pairs):
    return torch.tensor([10000.0 ** (-i / n) for n in pairs for i in range(n)], dtype=torch.float32, device="cuda")


def rotary_bound(x, want, heads, P, interleaved):
    """Sine and cosine: the reduced angle and the functions, 2^-21 of 1; two
    products and a sum, 4 roundings of the pair's length; one rounding of the output."""
    B, L, C = x.shape
    y = x.double().reshape(B, L, heads, -1)
    i1 = torch.arange(P, device=x.device) * (2 if interleaved else 1)
    i2 = i1 + (1 if interleaved else P)
    n = torch.zeros_like(y)
    n[..., i1] = n[..., i2] = y[..., i1].abs() + y[..., i2].abs()
    return n.reshape(B, L, C) * (2.0 ** -21 + 4 * ref.F32_STEP) + ref.step(x.dtype) * want.abs()


# B, (T, H, W), heads, kv_heads, d, pairs
ROTARY = [
    (2, (1, 7, 7), 2, 2, 32, (0, 8, 8)), (1, (1, 1, 1), 1, 1, 32, (4, 6, 6)), (3, (4, 5, 3), 4, 2, 64, (8, 12, 12)),
    (2, (1, 9, 11), 3, 1, 32, (0, 5, 6)), (1, (2, 3, 5), 2, 2, 128, (30, 17, 17)), (1, (300, 1, 1), 8, 2, 64, (32, 0, 0)),
    (2, (1, 33, 1), 1, 1, 8, (0, 3, 0)), (1, (2, 2, 2), 1, 1, 512, (100, 100, 56)), (2, (3, 16, 17), 16, 4, 24, (2, 1, 1)),
]


# pairs that are no whole vectors: many heads, vectors that hold both halves' ends, head sizes that divide no
# CTA, more than one pass
ROTARY += [(2, (2, 13, 17), 6, 3, 24, (3, 2, 4)), (1, (1, 40, 9), 5, 5, 40, (5, 5, 5)), (3, (4, 7, 9), 9, 1, 64, (13, 9, 9)),
           (1, (1, 3, 2), 2, 1, 512, (100, 100, 51)), (40, (1, 56, 56), 2, 2, 32, (5, 5, 5)), (2, (1, 5, 7), 1, 1, 32, (1, 0, 0))]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("case", ROTARY, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}x{c[4]}")
def test_rotary_matches_the_definition(case, interleaved, dtype):
    B, grid, h, kv, d, pairs = case
    L, t = math.prod(grid), T[dtype]
    q, k = tokens(1, B, L, h * d, dtype=t), tokens(2, B, L, kv * d, dtype=t)
    f = freqs(pairs)
    own = torch.randint(-200000, 200000, (B, L, 3), device="cuda", dtype=torch.int32,
                        generator=torch.Generator(device="cuda").manual_seed(3))
    for pos in (None, own, own[:1].contiguous()):
        for inverse in (False, True):
            s = bra.rotary_shape_for(q, k, h, kv, pairs, grid=grid, pos=pos, interleaved=interleaved, inverse=inverse)
            (qo, iq), (ko, ik) = guarded(q.shape, t), guarded(k.shape, t)
            bra.bra_rotary(s, q, k, pos, f, qo, ko)
            assert iq() and ik()
            at = ref.grid_positions(*grid, "cuda") if pos is None else pos
            for x, y, n in ((q, qo, h), (k, ko, kv)):
                want = ref.rotary(x, n, pairs, f, at, interleaved, inverse)
                err = (y.double() - want).abs()
                assert bool((err <= rotary_bound(x, want, n, sum(pairs), interleaved)).all()), float(err.max())
                rest = y.view(B, L, n, d)[..., 2 * sum(pairs):]
                assert torch.equal(rest, x.view(B, L, n, d)[..., 2 * sum(pairs):])


def test_rotary_far_positions():
    """Positions over the whole int32 range: the angle is formed in 64 bits."""
    pos = torch.tensor([[[2 ** 31 - 1, -2 ** 31, 123456789]]], dtype=torch.int32, device="cuda")
    q, f = tokens(1, 1, 1, 32, dtype=torch.float32), freqs((4, 6, 6))
    s = bra.rotary_shape_for(q, None, 1, 0, (4, 6, 6), pos=pos)
    out = torch.empty_like(q)
    bra.bra_rotary(s, q, None, pos, f, out, None)
    want = ref.rotary(q, 1, (4, 6, 6), f, pos)
    # fp64 turns of 2^31 radians are good to 2^-22 of a turn, on both sides
    assert float((out.double() - want).abs().max()) <= float(q.abs().max()) * (2.0 ** -18 + 2.0 ** -20)


@pytest.mark.parametrize("pairs", [(0, 8, 8), (0, 7, 6)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotary_in_place_slices_and_inverse(dtype, pairs):
    t, f = T[dtype], freqs(pairs)
    wide = tokens(1, 2, 49, 3 * 64, dtype=t)  # a projection's q | k | v
    keep = wide.clone()
    q, k = wide[..., :64], wide[..., 64:128]
    s = bra.rotary_shape_for(q, k, 2, 2, pairs, grid=(1, 7, 7), q_out=q, k_out=k)
    dense = bra.rotary_shape_for(q, k, 2, 2, pairs, grid=(1, 7, 7))
    a, b = torch.empty((2, 49, 64), dtype=t, device="cuda"), torch.empty((2, 49, 64), dtype=t, device="cuda")
    bra.bra_rotary(dense, q, k, None, f, a, b)
    bra.bra_rotary(s, q, k, None, f, q, k)
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(wide[..., 128:], keep[..., 128:])
    # <rotated x, y> = <x, y turned back>: the inverse is the gradient
    y = tokens(2, 2, 49, 64, dtype=t)
    inv = bra.rotary_shape_for(y, None, 2, 0, pairs, grid=(1, 7, 7), inverse=True)
    back = torch.empty_like(y)
    bra.bra_rotary(inv, y, None, None, f, back, None)
    lhs, rhs = (a.double() * y.double()).sum(), (keep[..., :64].double() * back.double()).sum()
    n = float((a.double().abs() * y.double().abs()).square().sum().sqrt())
    assert abs(float(lhs - rhs)) <= 8 * 2 * (ref.step(t) + 2.0 ** -20) * n


def test_rotary_of_nothing():
    q = torch.empty((0, 5, 64), device="cuda")
    bra.bra_rotary(bra.rotary_shape_for(q, None, 2, 0, (16, 0, 0)), q, None, None, freqs((16, 0, 0)), q, None)


# n as a shape, unit
DROPS = [((1,), 1), ((7,), 1), ((8,), 1), ((3, 5, 32), 1), ((2, 49, 64), 64), ((4, 9, 96), 9 * 96), ((1000, 33), 1),
         ((3, 7, 8), 8), ((5, 13), 24)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape,unit", DROPS, ids=str)
def test_dropout_matches_the_definition(shape, unit, dtype):
    t, n = T[dtype], math.prod(shape)
    x, r = tokens(1, *shape, dtype=t), tokens(2, *shape, dtype=t)
    for p, seed, offset in ((0.0, 1, 0), (0.1, 2 ** 63 + 5, 2 ** 32 - 3), (0.5, 7, 2 ** 64 - 2), (1.0, 3, 9)):
        rng = torch.tensor([seed - 2 ** 64 if seed >= 2 ** 63 else seed,
                            offset - 2 ** 64 if offset >= 2 ** 63 else offset], dtype=torch.int64, device="cuda")
        keep = ref.keeps(n, unit, p, seed, offset).cuda().view(shape)
        dirty = torch.where(keep, x, torch.tensor(float("nan"), dtype=t, device="cuda"))  # dropped: anything
        scale = 1.0 / (1.0 - p) if p < 1 else 0.0
        for res in (r, None):
            y, intact = guarded(shape, t)
            bra.bra_dropout_add(dirty, res, p, rng, y, unit=unit)
            assert intact()
            want = torch.where(keep, x.double() * scale, 0.0) + (0.0 if res is None else res.double())
            err = (y.double() - want).abs()
            # 1 / (1 - p) and the multiply-add in fp32, one rounding of the output
            bound = 2 * ref.F32_STEP * (x.double().abs() * scale + want.abs()) + ref.step(t) * want.abs()
            assert bool((err <= bound * 1.01).all()), float(err.max())


def test_dropout_in_place_gradient_and_graph():
    """y over x or the residual; the gradient's mask is the forward's; a graph
    that reads a new offset draws a new mask."""
    x, r = tokens(1, 2, 77, 64, dtype=torch.bfloat16), tokens(2, 2, 77, 64, dtype=torch.bfloat16)
    rng = torch.tensor([11, 5], dtype=torch.int64, device="cuda")
    y = torch.empty_like(x)
    bra.bra_dropout_add(x, r, 0.3, rng, y)
    for into in (0, 1):
        a = [x.clone(), r.clone()]
        bra.bra_dropout_add(a[0], a[1], 0.3, rng, a[into])
        assert torch.equal(a[into], y)
    one = torch.ones_like(x)
    g, kept = torch.empty_like(x), torch.empty_like(x)
    bra.bra_dropout_add(one, None, 0.3, rng, g)
    bra.bra_dropout_add(x, None, 0.3, rng, kept)
    assert torch.equal(g != 0, ref.keeps(x.numel(), 1, 0.3, 11, 5).cuda().view(x.shape))
    assert torch.equal(kept != 0, (g != 0) & (x != 0))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        bra.bra_dropout_add(one, None, 0.3, rng, g)
    rng[1] = 1000
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g != 0, ref.keeps(x.numel(), 1, 0.3, 11, 1000).cuda().view(x.shape))


def test_dropout_past_32_bits():
    """More elements than 2^32 draws of one counter word: the far end's mask."""
    n = (1 << 32) + 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    rng = torch.tensor([3, 0], dtype=torch.int64, device="cuda")
    bra.bra_dropout_add(x, None, 0.5, rng, x)
    tail = ref.keeps(24, 1, 0.5, 3, 1 << 30)
    assert torch.equal((x[-24:] != 0).cpu(), tail)
    assert torch.equal((x[:24] != 0).cpu(), ref.keeps(24, 1, 0.5, 3, 0))

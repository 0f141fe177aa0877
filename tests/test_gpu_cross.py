"""Cross attention to an encoder's states (bra_cross_attend and its backward)
against the 64-bit definition, within bounds derived from the kernels'
roundings (block_reference.cross_bounds)."""
import math

import pytest
import torch

import block_reference as ref
import dynamic_sparse_attention_bra_b200 as bra
from parity import record_margin

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}


def tokens(seed, *shape, dtype, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") + mean).to(dtype)


def guarded(shape, dtype, fill=float("nan")):
    """A tensor between two bands of a fixed pattern, and a function that looks at them."""
    n, band = math.prod(shape), 4096
    e = torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((2 * band + -(-n * e // 16) * 16,), 0xA5, dtype=torch.uint8, device="cuda")
    t = buf[band:band + n * e].view(dtype).view(shape)
    t.fill_(fill)

    def intact():
        return bool((buf[:band] == 0xA5).all()) and bool((buf[band + n * e:] == 0xA5).all())
    return t, intact


def run(q, k, v, heads, kv_heads, kv_len=None, kv_mask=None, grad=None, scale=None, ws=None):
    s = bra.cross_shape_for(q, k, v, heads, kv_heads, scale)
    if ws is None:
        ws = torch.zeros(bra.bra_cross_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    o, io = guarded((s.B, s.Lq, heads * s.d), q.dtype)
    lse, il = guarded((s.B, heads, s.Lq), torch.float32)
    bra.bra_cross_attend(s, q, k, v, kv_len, kv_mask, o, lse, ws)
    out, checks = {"o": o, "lse": lse}, [io, il]
    if grad is not None:
        for name, n, h in (("dq", s.Lq, heads), ("dk", s.Lk, kv_heads), ("dv", s.Lk, kv_heads)):
            out[name], c = guarded((s.B, n, h * s.d), q.dtype)
            checks.append(c)
        bra.bra_cross_attend_backward(s, q, k, v, kv_len, kv_mask, o, lse, grad, out["dq"], out["dk"], out["dv"], ws)
    assert bra.bra_cross_device_status(s, ws) == bra.BRA_OK
    assert all(c() for c in checks), "written outside an output"
    return out


def check(name, out, q, k, v, heads, kv_heads, ok, grad=None, scale=None):
    r = ref.cross(q, k, v, heads, kv_heads, ok, scale, grad)
    b = ref.cross_bounds(r, q.dtype, q.shape[-1] // heads, k.shape[1], q.shape[1] * heads // kv_heads)
    for x, got in out.items():
        want = r[x].reshape(got.shape)
        fine = torch.isfinite(want)
        assert torch.equal(fine, torch.isfinite(got)) and torch.equal(want[~fine], got[~fine].double()), x
        ratio = ((got.double() - want).abs()[fine] / b[x].reshape(got.shape)[fine])
        worst = float(ratio.max()) if ratio.numel() else 0.0
        record_margin(f"cross {name} {x}", worst, 1.0)
        assert worst <= 1.0, f"{x}: {worst:.3f} of the bound"
        if q.dtype == torch.float32 and x != "lse":
            # the bound above takes every rounding at its worst; their mean square stays far below
            # a rounding to fewer bits (2^-11 for tf32), which it would let pass
            whole = r[{"o": "abs_o", "dq": "all_dq", "dk": "all_dk", "dv": "abs_dv"}[x]]
            assert float((got.double() - want).norm()) <= 2.0 ** -16 * float(whole.norm()), x


# B, Lq, Lk, heads, kv_heads, d: one token to long, odd sizes, every head size, groups, split states
SIZES = [
    (1, 1, 1, 1, 1, 32), (1, 1, 49, 2, 2, 32), (3, 1, 700, 4, 1, 64), (2, 3, 2049, 8, 2, 128), (1, 16, 5000, 1, 1, 32),
    (2, 17, 63, 2, 2, 32), (2, 49, 64, 3, 3, 64), (1, 130, 65, 4, 2, 128), (2, 197, 127, 6, 2, 32),
    (1, 784, 196, 4, 4, 32), (2, 333, 1025, 2, 1, 64), (1, 257, 4500, 2, 2, 128), (1, 64, 3000, 12, 3, 32),
    (5, 300, 300, 8, 8, 64), (1, 513, 385, 16, 4, 128), (2, 9, 16, 32, 4, 32),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("valid", ["all", "len", "mask", "both"])
def test_matches_the_definition(size, dtype, valid):
    B, Lq, Lk, h, kv, d = size
    t = T[dtype]
    q, g = tokens(1, B, Lq, h * d, dtype=t), tokens(4, B, Lq, h * d, dtype=t)
    k, v = tokens(2, B, Lk, kv * d, dtype=t, mean=0.5), tokens(3, B, Lk, kv * d, dtype=t, mean=0.3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = m = None
    if valid in ("len", "both"):
        n = torch.randint(0, Lk + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        n[-1] = Lk if B == 1 else 0  # an entry without states
        n[0] = max(1, Lk - 1)
    if valid in ("mask", "both"):
        m = (torch.rand((B, Lk), generator=gen, device="cuda") < 0.6).to(torch.uint8) * 255
    ok = ref.valid_states(B, Lk, n, m, "cuda")
    # whatever lies in masked places stays out of the results
    junk = torch.where(torch.arange(Lk, device="cuda") % 2 == 0, float("nan"), float("inf"))[None, :, None].to(t)
    k2, v2 = (torch.where(ok[:, :, None], x, junk) for x in (k, v))
    out = run(q, k2, v2, h, kv, n, m, g)
    check(f"{dtype} {valid} {size}", out, q, k, v, h, kv, ok, g)


# many more units of work than SMs, groups that divide no tile, last tiles of one row, long states
MANY = [(40, 600, 300, 4, 4, 32), (60, 300, 400, 2, 2, 64), (24, 400, 333, 6, 6, 128), (3, 200, 700, 6, 2, 64),
        (2, 150, 300, 3, 1, 128), (1, 1100, 1300, 5, 1, 32), (2, 513, 2500, 2, 2, 32), (1, 129, 4097, 2, 2, 64),
        (5, 1025, 257, 2, 1, 32), (70, 49, 100, 4, 4, 32), (9, 260, 256, 8, 2, 64)]
# as many scores as the many-row forms take, in units that end inside a tile; long splits
MANY += [(3, 1030, 2900, 6, 2, 32), (1, 131, 33000, 4, 4, 32), (70, 129, 501, 4, 4, 32), (1, 4099, 1025, 4, 4, 32),
         (3, 211, 1700, 6, 2, 64), (1, 129, 17001, 2, 2, 64), (9, 700, 256, 8, 2, 64), (40, 300, 90, 2, 2, 64),
         (2, 450, 2300, 6, 2, 128), (1, 128, 33000, 1, 1, 128), (60, 129, 65, 9, 9, 128), (1, 2000, 513, 5, 5, 128)]


@pytest.mark.parametrize("valid", ["all", "both"])
@pytest.mark.parametrize("size", MANY, ids=lambda s: "x".join(map(str, s)))
def test_many_units_and_odd_groups(size, valid):
    test_matches_the_definition(size, "bf16", valid)


@pytest.mark.parametrize("Lq", [70, 9400])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores_and_scale(dtype, Lq):
    """A running maximum that keeps rising, sums dominated by one state, another scale."""
    B, Lk, h, d = 1, 900, 2, 32
    q, g = tokens(1, B, Lq, h * d, dtype=T[dtype]), tokens(4, B, Lq, h * d, dtype=T[dtype])
    k, v = tokens(2, B, Lk, h * d, dtype=T[dtype]), tokens(3, B, Lk, h * d, dtype=T[dtype])
    k = (k.float() * torch.linspace(0.01, 12, Lk, device="cuda")[None, :, None]).to(T[dtype])
    ok = ref.valid_states(B, Lk, device="cuda")
    check(f"rising {dtype} {Lq}", run(q, k, v, h, h, grad=g, scale=0.3), q, k, v, h, h, ok, g, 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Lq,heads", [(300, 4), (1, 4), (450, 4)])
def test_slices_and_shared_states(dtype, Lq, heads):
    """K and V as halves of one projection, Q a slice of a wider tensor, states
    that all entries share (a batch step of 0): results as from dense copies."""
    B, Lk, kv, d, t = 3, 1100, 2, 64, T[dtype]
    wide, kvp = tokens(1, B, Lq, heads * d + 64, dtype=t), tokens(2, 1, Lk, 2 * kv * d, dtype=t).expand(B, -1, -1)
    q, k, v = wide[..., 32:32 + heads * d], kvp[..., :kv * d], kvp[..., kv * d:]
    assert not q.is_contiguous() or Lq == 1
    g = tokens(4, B, Lq, heads * d, dtype=t)
    a = run(q, k, v, heads, kv, grad=g)
    b = run(q.contiguous(), k.contiguous(), v.contiguous(), heads, kv, grad=g)
    assert all(torch.equal(a[x], b[x]) for x in a)
    check(f"slices {dtype} {Lq}", a, q, k, v, heads, kv, ref.valid_states(B, Lk, device="cuda"), g)


def test_offsets_past_32_bits():
    """Entries more than 2^32 bytes (and 2^31 elements) apart in a cache."""
    step = (1 << 31) + 4096
    buf = torch.empty(step + 64 * 600 * 2, dtype=torch.bfloat16, device="cuda")
    kv = buf.as_strided((2, 600, 128), (step, 128, 1))
    small = tokens(2, 2, 600, 128, dtype=torch.bfloat16)
    kv[0].copy_(small[0])
    kv[1].copy_(small[1])
    for Lq in (1, 200, 1800):
        q, g = tokens(1, 2, Lq, 64, dtype=torch.bfloat16), tokens(3, 2, Lq, 64, dtype=torch.bfloat16)
        a = run(q, kv[..., :64], kv[..., 64:], 2, 2, grad=g)
        b = run(q, small[..., :64].contiguous(), small[..., 64:].contiguous(), 2, 2, grad=g)
        assert all(torch.equal(a[x], b[x]) for x in a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_states_and_no_tokens(dtype):
    t = T[dtype]
    q, g = tokens(1, 2, 70, 64, dtype=t), tokens(2, 2, 70, 64, dtype=t)
    none = torch.empty((2, 0, 64), dtype=t, device="cuda")
    out = run(q, none, none, 2, 2, grad=g)
    assert float(out["o"].float().abs().max()) == 0 and bool((out["lse"] == -math.inf).all())
    assert float(out["dq"].float().abs().max()) == 0
    k = tokens(3, 2, 90, 64, dtype=t)
    empty = torch.empty((2, 0, 64), dtype=t, device="cuda")
    out = run(empty, k, k, 2, 2, grad=empty)
    assert float(out["dk"].float().abs().max()) == 0 and float(out["dv"].float().abs().max()) == 0


def test_lengths_are_clamped():
    q, k = tokens(1, 3, 40, 64, dtype=torch.bfloat16), tokens(2, 3, 90, 64, dtype=torch.bfloat16)
    a = run(q, k, k, 2, 2, torch.tensor([-5, 1000, 90], dtype=torch.int32, device="cuda"))
    b = run(q, k, k, 2, 2, torch.tensor([0, 90, 90], dtype=torch.int32, device="cuda"))
    assert all(torch.equal(a[x], b[x]) for x in a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Lq,Lk", [(1, 6000), (400, 300), (2300, 2000)])
def test_same_bits_again(dtype, Lq, Lk):
    q, g = tokens(1, 2, Lq, 128, dtype=T[dtype]), tokens(4, 2, Lq, 128, dtype=T[dtype])
    k, v = tokens(2, 2, Lk, 64, dtype=T[dtype]), tokens(3, 2, Lk, 64, dtype=T[dtype])
    a, b = (run(q, k, v, 4, 2, grad=g) for _ in range(2))
    assert all(torch.equal(a[x], b[x]) for x in a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_match_differences(dtype):
    """sum(o g) moves by <dq, e> when q moves by e, measured on the kernel's own outputs."""
    t = T[dtype]
    x = [tokens(i, 1, n, 64, dtype=t) for i, n in ((1, 96), (2, 150), (3, 150))]
    g = tokens(4, 1, 96, 64, dtype=t)
    out = run(*x, 2, 2, grad=g)
    for i, name in enumerate(("dq", "dk", "dv")):
        e = tokens(10 + i, *x[i].shape, dtype=torch.float32).double()
        h = 2.0 ** -5
        ends = []
        for sign in (1, -1):
            y = list(x)
            y[i] = (x[i].double() + sign * h * e).to(t)
            ends.append((run(*y, 2, 2)["o"].double(), y[i].double()))
        moved = ends[0][1] - ends[1][1]  # what the type kept of the step
        seen = float(((ends[0][0] - ends[1][0]) * g.double()).sum())
        want = float((out[name].double() * moved).sum())
        # o's roundings: independent, half a step of each of its elements at both ends, six deviations;
        # third derivatives of the softmax: h^2 of the change, with room
        r = ref.step(t) * float((ends[0][0].abs() * g.double().abs()).square().sum().sqrt()) * 2 ** 0.5 * 6
        r += ref.step(t) * float((out[name].double().abs() * moved.abs()).square().sum().sqrt()) * 6
        assert abs(seen - want) <= r + 4 * h * h * float((out[name].double() * moved).abs().sum()) + 1e-5


def test_replayed_graphs_that_share_a_workspace():
    """Two captured forms (a token over long states, a training step), one
    workspace, replayed in turn on new inputs, on a stream of its own."""
    dt = torch.bfloat16
    k, v = (tokens(i, 2, 3000, 64, dtype=dt) for i in (2, 3))
    q1, q2, g = (tokens(i, 2, n, 128, dtype=dt) for i, n in ((1, 1), (4, 200), (5, 200)))
    s1, s2 = (bra.cross_shape_for(q, k, v, 4, 2) for q in (q1, q2))
    ws = torch.zeros(max(map(bra.bra_cross_workspace_bytes, (s1, s2))), dtype=torch.uint8, device="cuda")
    o1, o2 = torch.empty_like(q1), torch.empty_like(q2)
    lse = torch.empty((2, 4, 200), device="cuda")
    dq, dk, dv = torch.empty_like(q2), torch.empty_like(k), torch.empty_like(v)

    def first(stream=None):
        bra.bra_cross_attend(s1, q1, k, v, None, None, o1, None, ws, stream)

    def second(stream=None):
        bra.bra_cross_attend(s2, q2, k, v, None, None, o2, lse, ws, stream)
        bra.bra_cross_attend_backward(s2, q2, k, v, None, None, o2, lse, g, dq, dk, dv, ws, stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        first(side)
        second(side)
        for f in (first, second):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                f()
        for _ in range(2):
            for x in (q1, q2, k, v, g):
                x.normal_()
            for gr in graphs + graphs[:1]:
                gr.replay()
    side.synchronize()
    got = [x.clone() for x in (o1, o2, lse, dq, dk, dv)]
    first()
    second()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (o1, o2, lse, dq, dk, dv)))


def test_wrapper_on_a_map():
    """cross_attention on a map [B, H, W, C], two calls at once on two streams."""
    q, k = tokens(1, 2, 14, 14, 128, dtype=torch.bfloat16), tokens(2, 2, 77, 128, dtype=torch.bfloat16)
    o, lse = bra.cross_attention(q, k, k, 4)
    assert o.shape == q.shape and lse.shape == (2, 4, 196)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [bra.cross_attention(q, k, k, 4, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) and torch.equal(lse, b) for a, b in outs)
    with pytest.raises(bra.BraError):
        bra.cross_attention(q, k, k, 8)  # d = 16
    with pytest.raises(ValueError):
        bra.cross_attention(q, k.cpu(), k, 4)


# one size for every form of the kernels, forward and backward
FORMS = [(2, 3, 600, 4, 2, 32), (2, 40, 300, 4, 2, 128), (3, 200, 77, 2, 2, 32), (40, 250, 100, 2, 2, 64),
         (20, 600, 400, 4, 4, 32), (6, 513, 700, 4, 2, 64), (3, 600, 900, 4, 4, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", FORMS, ids=lambda s: "x".join(map(str, s)))
def test_a_token_that_is_not_finite_stays_with_its_own(size, dtype):
    """NaN in one token's Q and infinities in its gradient: the other tokens' o, lse and dq, and
    all of the other entries' gradients, keep their bits; invalid states still get zeros."""
    B, Lq, Lk, h, kv, d = size
    t = T[dtype]
    q, g = tokens(1, B, Lq, h * d, dtype=t), tokens(4, B, Lq, h * d, dtype=t)
    k, v = tokens(2, B, Lk, kv * d, dtype=t), tokens(3, B, Lk, kv * d, dtype=t)
    m = (torch.rand((B, Lk), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda") < 0.7).to(torch.uint8)
    n = torch.full((B,), Lk - 1, dtype=torch.int32, device="cuda")
    ok = ref.valid_states(B, Lk, n, m, "cuda")
    a = run(q, k, v, h, kv, n, m, g)
    q2, g2 = q.clone(), g.clone()
    q2[1, Lq // 2, 5], g2[1, Lq // 2] = float("nan"), float("inf")
    b = run(q2, k, v, h, kv, n, m, g2)
    others = torch.ones((B, Lq), dtype=torch.bool, device="cuda")
    others[1, Lq // 2] = False
    for x in ("o", "dq"):
        assert torch.equal(a[x][others], b[x][others]), x
    assert torch.equal(a["lse"].transpose(1, 2)[others], b["lse"].transpose(1, 2)[others])
    for x in ("dk", "dv"):
        assert torch.equal(a[x][0], b[x][0]) and torch.equal(a[x][2:], b[x][2:]), x
        assert float(b[x][~ok].float().abs().max()) == 0, x


def test_a_stream_s_memory_is_its_own():
    """The wrapper's workspace, freed as it returns, is not handed out again under its kernels."""
    q, k = tokens(1, 2, 300, 256, dtype=torch.bfloat16), tokens(2, 2, 6000, 256, dtype=torch.bfloat16)
    o, lse = bra.cross_attention(q, k, k, 8)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        o2, lse2 = bra.cross_attention(q, k, k, 8, stream=stream)
        junk = [torch.full((1 << 21,), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and len(junk) == 8


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", FORMS, ids=lambda s: "x".join(map(str, s)))
def test_an_entry_without_states_gets_zeros_from_any_gradient(size, dtype):
    B, Lq, Lk, h, kv, d = size
    t = T[dtype]
    q, g = tokens(1, B, Lq, h * d, dtype=t), tokens(4, B, Lq, h * d, dtype=t)
    k, v = tokens(2, B, Lk, kv * d, dtype=t), tokens(3, B, Lk, kv * d, dtype=t)
    m = torch.ones((B, Lk), dtype=torch.bool, device="cuda")
    m[0] = False
    g[0, Lq // 2], g[0, 0, 1] = float("inf"), float("nan")
    out = run(q, k, v, h, kv, None, m, g)
    assert bool((out["lse"][0] == -math.inf).all())
    assert all(float(out[x][0].float().abs().max()) == 0 for x in ("o", "dq", "dk", "dv"))
    assert all(bool(torch.isfinite(out[x][1:]).all()) for x in out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", FORMS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("spans", ["left", "hole", "last"])
def test_masks_of_whole_blocks(size, dtype, spans):
    """Padding on the left, invalid stretches longer than any block, one valid state at the very end."""
    B, Lq, Lk, h, kv, d = size
    t = T[dtype]
    q, g = tokens(1, B, Lq, h * d, dtype=t), tokens(4, B, Lq, h * d, dtype=t)
    k, v = tokens(2, B, Lk, kv * d, dtype=t, mean=0.5), tokens(3, B, Lk, kv * d, dtype=t, mean=0.3)
    m = torch.zeros((B, Lk), dtype=torch.uint8, device="cuda")
    for b in range(B):
        if spans == "left":
            m[b, min(Lk - 1, (b + 1) * Lk // (B + 1)):] = 1
        elif spans == "hole":
            m[b, : 1 + b % 3] = 1
            m[b, Lk - 1 - b % 5:] = 1
        else:
            m[b, -1] = 1
    ok = ref.valid_states(B, Lk, None, m, "cuda")
    k2, v2 = (torch.where(ok[:, :, None], x, float("nan")) for x in (k, v))
    check(f"spans {spans} {dtype} {size}", run(q, k2, v2, h, kv, None, m, g), q, k, v, h, kv, ok, g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", FORMS, ids=lambda s: "x".join(map(str, s)))
def test_scores_far_from_zero(size, dtype):
    """Scores around +-3000: the first states far below the last, and all of them far below zero."""
    B, Lq, Lk, h, kv, d = size
    t = T[dtype]
    k, v = torch.ones((B, Lk, kv * d), device="cuda"), tokens(3, B, Lk, kv * d, dtype=t)
    k = (k * torch.linspace(-30, 30, Lk, device="cuda")[None, :, None]).to(t)
    for sign in (1.0, -1.0):
        q = torch.full((B, Lq, h * d), sign * 100 / d, device="cuda").to(t)
        out = run(q, k, v, h, kv, scale=1.0)
        check(f"far {dtype} {size} {sign}", out, q, k, v, h, kv, ref.valid_states(B, Lk, device="cuda"), None, 1.0)
        out = run(q, (k.float() - 30.5 * sign).to(t), v, h, kv, scale=1.0)
        assert bool(torch.isfinite(out["o"]).all()) and float(out["lse"].max()) < 0

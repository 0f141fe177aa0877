"""What cross attention says of a token whose sums are not finite: NaN in its own o, lse
and gradients, in every form of the kernels; -infinity stays the log sum of a token
without valid states."""
import math

import pytest
import torch

import block_reference as ref
from test_gpu_cross import FORMS, T, run, tokens

pytestmark = pytest.mark.gpu

# and the forms whose states are split over CTAs
SIZES = FORMS + [(2, 1, 3000, 2, 1, 64), (2, 200, 2100, 4, 4, 64), (2, 450, 2300, 6, 2, 128), (2, 1030, 2900, 6, 2, 32)]


def inputs(size, dtype):
    B, Lq, Lk, h, kv, d = size
    t = T[dtype]
    q, g = tokens(1, B, Lq, h * d, dtype=t), tokens(4, B, Lq, h * d, dtype=t)
    k, v = tokens(2, B, Lk, kv * d, dtype=t), tokens(3, B, Lk, kv * d, dtype=t)
    gen = torch.Generator(device="cuda").manual_seed(5)
    m = (torch.rand((B, Lk), generator=gen, device="cuda") < 0.7).to(torch.uint8)
    m[:, Lk // 2] = 1
    m[0] = 0
    return q, k, v, g, m, ref.valid_states(B, Lk, None, m, "cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_query_with_nan(size, dtype):
    B, Lq, Lk, h, kv, d = size
    q, k, v, g, m, ok = inputs(size, dtype)
    at = Lq // 2
    q[:, at, 5] = float("nan")  # head 0, which reads state head 0
    out = run(q, k, v, h, kv, None, m, g)
    nan = torch.zeros((B, Lq, h), dtype=torch.bool, device="cuda")
    nan[1:, at, 0] = True
    for x in ("o", "dq"):
        assert torch.equal(out[x].view(B, Lq, h, d).isnan(), nan[..., None].expand(-1, -1, -1, d)), x
    assert torch.equal(out["lse"].isnan(), nan.transpose(1, 2))
    assert bool((out["lse"][0] == -math.inf).all()) and bool(torch.isfinite(out["lse"][1:][~nan.transpose(1, 2)[1:]]).all())
    # every valid state of head 0 has a NaN in its sums, the other heads' states none
    bad = torch.zeros((B, Lk, kv), dtype=torch.bool, device="cuda")
    bad[..., 0] = ok
    for x in ("dk", "dv"):
        assert torch.equal(out[x].view(B, Lk, kv, d).isnan(), bad[..., None].expand(-1, -1, -1, d)), x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_valid_key_with_nan(size, dtype):
    """All tokens that read it have a NaN among their scores."""
    B, Lq, Lk, h, kv, d = size
    q, k, v, g, m, ok = inputs(size, dtype)
    k[:, Lk // 2, d - 1] = float("nan")  # state head 0
    out = run(q, k, v, h, kv, None, m, g)
    nan = torch.zeros((B, Lq, h), dtype=torch.bool, device="cuda")
    nan[1:, :, :h // kv] = True
    for x in ("o", "dq"):
        assert torch.equal(out[x].view(B, Lq, h, d).isnan(), nan[..., None].expand(-1, -1, -1, d)), x
    assert torch.equal(out["lse"].isnan(), nan.transpose(1, 2))
    assert bool((out["lse"][0] == -math.inf).all())


@pytest.mark.parametrize("value", [float("inf"), -3.4028e38])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_value_past_what_fp32_can_split_stays_in_its_channel(size, dtype, value):
    """In fp32 such a value's parts make NaN, in bf16 the sums follow IEEE; either way the other
    channels, heads and entries keep their bits, and so does lse."""
    B, Lq, Lk, h, kv, d = size
    q, k, v, g, m, ok = inputs(size, dtype)
    a = run(q, k, v, h, kv, None, m)
    v2 = v.clone()
    v2[1, Lk // 2, 3] = value
    b = run(q, k, v2, h, kv, None, m)
    touched = torch.zeros((B, Lq, h, d), dtype=torch.bool, device="cuda")
    touched[1, :, :h // kv, 3] = True
    x, y = (t["o"].view(B, Lq, h, d) for t in (a, b))
    assert torch.equal(x[~touched], y[~touched]) and torch.equal(a["lse"], b["lse"])
    if dtype == "f32":
        assert bool(y[touched].isnan().all())
    elif math.isinf(value):
        assert not bool(torch.isfinite(y[touched]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_an_infinite_key_s_tokens_say_nan(size, dtype):
    """Scores of +-infinity: NaN where they are +infinity, nothing of the state
    where they are -infinity (NaN in fp32, whose parts know no infinity)."""
    B, Lq, Lk, h, kv, d = size
    q, k, v, g, m, ok = inputs(size, dtype)
    k[:, Lk // 2, 0] = float("inf")
    up = (q.view(B, Lq, h, d)[..., :h // kv, 0] > 0)
    out = run(q, k, v, h, kv, None, m)
    lse = out["lse"][:, :h // kv].transpose(1, 2)[1:]
    if dtype == "f32":
        assert bool(lse.isnan().all())
    else:
        assert torch.equal(lse.isnan(), up[1:])
        m2 = m.clone()
        m2[:, Lk // 2] = 0
        other = run(q, k, v, h, kv, None, m2)
        down = ~up[1:]
        assert bool((lse[down] - other["lse"][:, :h // kv].transpose(1, 2)[1:][down]).abs().max() <= 1e-3)
    assert bool((out["lse"][0] == -math.inf).all())

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

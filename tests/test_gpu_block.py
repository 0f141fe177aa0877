"""The operators together, as a conditioned block runs them: projection, rotary
positions, routed attention, dropout and residual, cross attention to an
encoder's states, dropout and residual; then the gradients back through it.
Each stage is compared with its 64-bit definition on the values that it read."""
import numpy as np
import pytest
import torch

import block_reference as ref
import dynamic_sparse_attention_bra_b200 as bra
import oracle
from test_gpu_cross import check, tokens

pytestmark = pytest.mark.gpu


def test_conditioned_block_forward_and_backward():
    B, H, W, C, heads, S, topk, Lk, p = 3, 28, 28, 64, 2, 7, 4, 53, 0.2
    dt, N = torch.bfloat16, H * W
    x, w = tokens(1, B, H, W, C, dtype=dt), (tokens(2, 3 * C, C, dtype=torch.float32) * C ** -0.5).to(dt)
    states = tokens(3, B, Lk, 2 * C, dtype=dt)  # projected keys | values of the encoder
    lens = torch.tensor([Lk, 0, 17], dtype=torch.int32, device="cuda")
    f = torch.tensor([100.0 ** (-i / 8) for i in range(8)] * 2, device="cuda")
    rng = [torch.tensor([42, i * 10 ** 6], dtype=torch.int64, device="cuda") for i in range(2)]
    shape = bra.shape_for(B, H, W, C, heads, S, topk, "bf16")
    ws = torch.zeros(bra.bra_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    new = lambda: torch.empty((B, H, W, C), dtype=dt, device="cuda")
    q, k, v, qt, kt, o, y, o2, z = (new() for _ in range(9))
    qr, kr = (torch.empty((B, heads, S * S, 32), device="cuda") for _ in range(2))
    idx = torch.empty((B, heads, S * S, topk), dtype=torch.int32, device="cuda")

    bra.bra_qkv_project(shape, x, w, None, q, k, v, qr, kr, ws)
    rs = bra.rotary_shape_for(q, k, heads, heads, (0, 8, 8), grid=(1, H, W))
    bra.bra_rotary(rs, q, k, None, f, qt, kt)
    bra.bra_route(shape, qt, kt, idx, ws)
    bra.bra_attend(shape, qt, kt, v, idx, o, ws)
    bra.bra_dropout_add(o, x, p, rng[0], y)
    ck, cv = states[..., :C], states[..., C:]
    cs = bra.cross_shape_for(y, ck, cv, heads)
    cws = torch.zeros(bra.bra_cross_workspace_bytes(cs), dtype=torch.uint8, device="cuda")
    lse = torch.empty((B, heads, N), device="cuda")
    bra.bra_cross_attend(cs, y, ck, cv, lens, None, o2, lse, cws)
    bra.bra_dropout_add(o2, y, p, rng[1], z, unit=N * C)  # stochastic depth
    assert bra.bra_device_status(shape, ws) == bra.BRA_OK

    flat = lambda t: t.reshape(B, N, C)
    at = ref.grid_positions(1, H, W, "cuda")
    for a, b in ((q, qt), (k, kt)):
        want = ref.rotary(flat(a), heads, (0, 8, 8), f, at)
        n = float(a.double().abs().max()) * 2
        assert bool(((flat(b).double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * n).all())
    f64 = lambda t: t.double().cpu().numpy()
    ro = oracle.token_attention(f64(qt), f64(kt), f64(v), idx.cpu().numpy(), heads, S)
    assert float(np.abs(f64(o) - ro).max()) <= 2e-2
    keep0 = ref.keeps(x.numel(), 1, p, 42, 0).cuda().view(x.shape)
    want = torch.where(keep0, o.double() / (1 - p), 0.0) + x.double()
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -21 * o.double().abs()).all())
    keep1 = ref.keeps(x.numel(), N * C, p, 42, 10 ** 6).cuda().view(x.shape)
    want = torch.where(keep1, o2.double() / (1 - p), 0.0) + y.double()
    assert bool(((z.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -21 * o2.double().abs()).all())

    # back: dz -> the depth's mask -> cross attention -> y's gradient -> dropout -> routed attention -> rotation
    dz = tokens(9, B, H, W, C, dtype=dt)
    do2, dq2, do = new(), new(), new()
    bra.bra_dropout_add(dz, None, p, rng[1], do2, unit=N * C)
    dk2, dv2 = (torch.empty((B, Lk, C), dtype=dt, device="cuda") for _ in range(2))
    bra.bra_cross_attend_backward(cs, y, ck, cv, lens, None, o2, lse, do2, dq2, dk2, dv2, cws)
    ok = ref.valid_states(B, Lk, lens, None, "cuda")
    check("block", {"o": flat(o2), "lse": lse, "dq": flat(dq2), "dk": dk2, "dv": dv2}, flat(y), ck, cv, heads, heads, ok,
          flat(do2))
    assert torch.equal(do2 != 0, keep1 & (dz != 0))
    dy = (dz.float() + dq2.float()).to(dt)
    bra.bra_dropout_add(dy, None, p, rng[0], do)
    gq, gk, gv = (torch.empty((B, H, W, C), device="cuda") for _ in range(3))
    bra.bra_attend_backward(shape, qt, kt, v, idx, do, gq, gk, gv, ws)
    assert bra.bra_device_status(shape, ws) == bra.BRA_OK
    assert bra.bra_cross_device_status(cs, cws) == bra.BRA_OK
    back = bra.rotary_shape_for(gq, gk, heads, heads, (0, 8, 8), grid=(1, H, W), inverse=True)
    dq, dk = torch.empty_like(gq), torch.empty_like(gk)
    bra.bra_rotary(back, gq, gk, None, f, dq, dk)
    for a, b in ((gq, dq), (gk, dk)):
        want = ref.rotary(flat(a), heads, (0, 8, 8), f, at, inverse=True)
        assert bool(((flat(b).double() - want).abs() <= 2.0 ** -20 * float(a.abs().max())).all())

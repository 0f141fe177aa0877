"""Orders of the operands that the other tests do not have: tokens first ([L, B, C]), entries
that overlap (a window that slides over one sequence), and rows far apart."""
import pytest
import torch

import dynamic_sparse_attention_bra_b200 as bra
from test_gpu_cross import FORMS, T, run, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", FORMS, ids=lambda s: "x".join(map(str, s)))
def test_tokens_first(size, dtype):
    B, Lq, Lk, h, kv, d = size
    t = T[dtype]
    q = tokens(1, Lq, B, h * d, dtype=t).transpose(0, 1)
    kvp = tokens(2, Lk, B, 2 * kv * d, dtype=t).transpose(0, 1)
    k, v, g = kvp[..., :kv * d], kvp[..., kv * d:], tokens(4, B, Lq, h * d, dtype=t)
    n = torch.tensor([Lk - b for b in range(B)], dtype=torch.int32, device="cuda")
    a = run(q, k, v, h, kv, n, None, g)
    b = run(q.contiguous(), k.contiguous(), v.contiguous(), h, kv, n, None, g)
    assert all(torch.equal(a[x], b[x]) for x in a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", FORMS, ids=lambda s: "x".join(map(str, s)))
def test_windows_that_slide(size, dtype):
    B, Lq, Lk, h, kv, d = size
    t = T[dtype]
    q, g = tokens(1, B, Lq, h * d, dtype=t), tokens(4, B, Lq, h * d, dtype=t)
    k, v = (tokens(i, 1, Lk + 3 * B, kv * d, dtype=t)[0].unfold(0, Lk, 3)[:B].transpose(1, 2) for i in (2, 3))
    assert k.shape == (B, Lk, kv * d) and k.stride() == (3 * kv * d, kv * d, 1)
    a = run(q, k, v, h, kv, None, None, g)
    b = run(q, k.contiguous(), v.contiguous(), h, kv, None, None, g)
    assert all(torch.equal(a[x], b[x]) for x in a)


@pytest.mark.parametrize("pairs", [(0, 8, 8), (0, 7, 6)], ids=str)
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotary_tokens_first(dtype, interleaved, pairs):
    B, L, t = 3, 35, T[dtype]
    q, k = (tokens(i, L, B, n * 32, dtype=t).transpose(0, 1) for i, n in ((1, 4), (2, 2)))
    qo, ko = (torch.empty((L, B, n * 32), dtype=t, device="cuda").transpose(0, 1) for n in (4, 2))
    f = torch.tensor([100.0 ** (-i / 8) for i in range(sum(pairs))], device="cuda")
    s = bra.rotary_shape_for(q, k, 4, 2, pairs, grid=(1, 5, 7), interleaved=interleaved, q_out=qo, k_out=ko)
    bra.bra_rotary(s, q, k, None, f, qo, ko)
    a, b = q.contiguous(), k.contiguous()
    x, y = torch.empty_like(a), torch.empty_like(b)
    bra.bra_rotary(bra.rotary_shape_for(a, b, 4, 2, pairs, grid=(1, 5, 7), interleaved=interleaved), a, b, None, f, x, y)
    assert torch.equal(qo, x) and torch.equal(ko, y)

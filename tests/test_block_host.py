"""Host side of the conditioned block's operators: every refusal happens before
any CUDA call (no kernel is launched by these tests), and shapes, strides and
workspace sizes follow from the tensors."""
import ctypes

import pytest
import torch

import dynamic_sparse_attention_bra_b200 as bra

P = 1 << 20  # a pointer that is never followed: the checks fail first
BAD, NO = bra.BRA_ERR_INVALID_ARG, bra.BRA_ERR_UNSUPPORTED


def cross_shape(**kw):
    a = dict(B=2, Lq=5, Lk=9, heads=4, kv_heads=2, d=32, dtype=bra.BRA_DTYPE_BF16, scale=0.5, q_row=128, q_batch=640,
             k_row=64, k_batch=576, v_row=64, v_batch=576)
    a.update(kw)
    return bra.BraCrossShape(*(a[f[0]] for f in bra.BraCrossShape._fields_))


def rotary_shape(**kw):
    a = dict(B=2, T=2, H=3, W=4, heads=4, kv_heads=2, d=32, pairs=(4, 6, 6), interleaved=0, inverse=0,
             dtype=bra.BRA_DTYPE_BF16, pos_batch=0, q_row=128, q_batch=24 * 128, k_row=64, k_batch=24 * 64, qo_row=128,
             qo_batch=24 * 128, ko_row=64, ko_batch=24 * 64)
    a.update(kw)
    return bra.BraRotaryShape(*(a[f[0]] for f in bra.BraRotaryShape._fields_))


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(Lq=-1), BAD), (dict(Lk=-2), BAD), (dict(heads=0), BAD), (dict(kv_heads=0), BAD),
    (dict(heads=3), BAD), (dict(d=0), BAD), (dict(dtype=2), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(q_row=120), BAD), (dict(q_row=129), BAD),
    (dict(k_row=32), BAD), (dict(v_row=-64), BAD), (dict(k_batch=4), BAD), (dict(v_batch=-8), BAD),
    (dict(d=16), NO), (dict(d=48), NO), (dict(d=256, q_row=1024, k_row=512, v_row=512), NO), (dict(B=65536), NO),
    (dict(Lk=(1 << 28) + 1), NO), (dict(Lq=1 << 27), NO),
])
def test_cross_shapes_refused(kw, code):
    s = cross_shape(**kw)
    assert bra.bra_cross_workspace_bytes(s) == 0
    r = ctypes.byref(s)
    assert bra._lib.bra_cross_attend(r, P, P, P, P, P, P, P, P, None) == code
    assert bra._lib.bra_cross_attend_backward(r, *([P] * 12), None) == code
    assert bra._lib.bra_cross_device_status(r, P, None) == code


def test_null_shapes_refused():
    assert bra._lib.bra_cross_attend(None, *([P] * 8), None) == BAD
    assert bra._lib.bra_cross_attend_backward(None, *([P] * 12), None) == BAD
    assert bra._lib.bra_rotary(None, *([P] * 6), None) == BAD


# order after the shape: q, k, v, kv_len, kv_mask, o, lse, workspace
@pytest.mark.parametrize("which,null_ok,off", [(0, False, 8), (1, False, 8), (2, False, 8), (3, True, 2), (5, False, 8),
                                               (6, True, 2), (7, False, 8)])
def test_cross_pointers_refused(which, null_ok, off):
    s = cross_shape()
    for bad in (P + off,) if null_ok else (0, P + off):
        a = [P] * 8
        a[which] = bad
        assert bra._lib.bra_cross_attend(ctypes.byref(s), *a, None) == BAD


# q, k, v, kv_len, kv_mask, o, lse, grad_o, dq, dk, dv, workspace
@pytest.mark.parametrize("which", [0, 1, 2, 5, 6, 7, 8, 9, 10, 11])
def test_cross_backward_pointers_refused(which):
    s = cross_shape()
    for bad in (0, P + 8):
        a = [P] * 12
        a[which] = bad
        assert bra._lib.bra_cross_attend_backward(ctypes.byref(s), *a, None) == BAD


def test_empty_cross_calls_do_nothing():
    for kw in (dict(B=0), dict(Lq=0)):
        s = cross_shape(**kw)
        assert bra.bra_cross_workspace_bytes(s) >= 256
        assert bra._lib.bra_cross_attend(ctypes.byref(s), None, P, P, None, None, None, None, P, None) == bra.BRA_OK
    s = cross_shape(B=0)
    assert bra._lib.bra_cross_attend_backward(ctypes.byref(s), *([None] * 11), P, None) == bra.BRA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(heads=0), BAD), (dict(kv_heads=0), BAD), (dict(d=0), BAD),
    (dict(dtype=3), BAD), (dict(pairs=(-1, 8, 8)), BAD), (dict(pairs=(0, 0, 0)), BAD), (dict(pairs=(6, 6, 6)), BAD),
    (dict(q_row=64), BAD), (dict(q_row=132), BAD), (dict(ko_row=32), BAD), (dict(k_batch=3), BAD),
    (dict(qo_batch=0), BAD), (dict(pos_batch=-3), BAD), (dict(d=20, pairs=(2, 2, 2)), NO),
    (dict(d=520, q_row=4096, k_row=4096, qo_row=4096, ko_row=4096), NO), (dict(B=70000), NO),
    (dict(T=1 << 10, H=1 << 10, W=1 << 10), NO),
])
def test_rotary_shapes_refused(kw, code):
    assert bra._lib.bra_rotary(ctypes.byref(rotary_shape(**kw)), P, 2 * P, None, P, 3 * P, 4 * P, None) == code


# q, k, pos, inv_freq, q_out, k_out
@pytest.mark.parametrize("which,bad", [(0, 0), (0, P + 8), (1, 0), (1, P + 8), (2, P + 2), (3, 0), (3, P + 1), (4, 0),
                                       (4, P + 4), (5, 0), (5, P + 4)])
def test_rotary_pointers_refused(which, bad):
    a = [P, 2 * P, None, P, 3 * P, 4 * P]
    a[which] = bad
    assert bra._lib.bra_rotary(ctypes.byref(rotary_shape()), *a, None) == BAD


def test_rotary_in_place_needs_equal_strides():
    s = rotary_shape(q_row=256, q_batch=24 * 256)
    assert bra._lib.bra_rotary(ctypes.byref(s), P, 2 * P, None, P, P, 4 * P, None) == BAD


@pytest.mark.parametrize("args,code", [
    ((2, 64, 1, 0.1), BAD), ((1, -1, 1, 0.1), BAD), ((1, 64, 0, 0.1), BAD), ((1, 64, 1, -0.1), BAD),
    ((1, 64, 1, 1.5), BAD), ((1, 64, 1, float("nan")), BAD), ((1, 64, 12, 0.1), NO), ((1, 1 << 41, 1, 0.1), NO),
])
def test_dropout_arguments_refused(args, code):
    assert bra._lib.bra_dropout_add(*args, P, P, P, P, None) == code


@pytest.mark.parametrize("which,bad", [(0, 0), (0, P + 4), (1, 0), (1, P + 8), (2, P + 8), (3, 0), (3, P + 8)])
def test_dropout_pointers_refused(which, bad):
    a = [P] * 4  # rng, x, residual, y
    a[which] = bad
    assert bra._lib.bra_dropout_add(1, 64, 1, 0.1, *a, None) == BAD


def test_dropout_of_nothing():
    assert bra._lib.bra_dropout_add(1, 0, 1, 0.1, P, None, None, None, None) == bra.BRA_OK


def test_cross_shape_from_tensors():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    s = bra.cross_shape_for(z(2, 7, 7, 64), z(2, 9, 32), z(2, 9, 32), 2, 1)  # a map's tokens
    assert (s.B, s.Lq, s.Lk, s.d, s.q_row, s.q_batch) == (2, 49, 9, 32, 64, 49 * 64)
    assert abs(s.scale - 32 ** -0.5) < 1e-7
    kv = z(2, 9, 128)
    s = bra.cross_shape_for(z(2, 5, 128), kv[..., :64], kv[..., 64:], 4, 2)  # two halves of one projection
    assert (s.k_row, s.k_batch, s.v_row, s.v_batch) == (128, 9 * 128, 128, 9 * 128)
    s = bra.cross_shape_for(z(3, 5, 128), z(1, 9, 64).expand(3, -1, -1), z(3, 9, 64), 4, 2)
    assert (s.k_batch, s.v_batch) == (0, 9 * 64)
    s = bra.cross_shape_for(z(1, 5, 256)[..., 128:], z(1, 1, 64), z(1, 1, 64), 4, 2)  # steps never taken are dense
    assert (s.q_row, s.q_batch, s.k_row, s.k_batch) == (256, 5 * 256, 64, 64)


def test_cross_shape_refuses_what_does_not_fit():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    for a in ((z(2, 5, 64), z(3, 9, 64), z(3, 9, 64), 2), (z(2, 5, 64), z(2, 9, 64), z(2, 8, 64), 2),
              (z(2, 5, 64), z(2, 9, 64).float(), z(2, 9, 64), 2), (z(2, 5, 64), z(2, 9, 96), z(2, 9, 64), 2),
              (z(2, 5, 64).half(), z(2, 9, 64), z(2, 9, 64), 2), (z(2, 64, 5).transpose(1, 2), z(2, 9, 64), z(2, 9, 64), 2),
              (z(2, 5, 65), z(2, 9, 64), z(2, 9, 64), 2)):
        with pytest.raises(ValueError):
            bra.cross_shape_for(*a)


def test_bindings_refuse_cpu_tensors_and_other_types():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    q, k = z(2, 5, 64), z(2, 9, 64)
    s = bra.cross_shape_for(q, k, k, 2)
    ws = torch.zeros(bra.bra_cross_workspace_bytes(s), dtype=torch.uint8)
    with pytest.raises(ValueError):
        bra.bra_cross_attend(s, q, k, k, None, None, z(2, 5, 64), None, ws)
    with pytest.raises(ValueError):
        bra.bra_cross_attend(s, q, k, k, None, None, z(2, 5, 64), None, ws[:128])
    with pytest.raises(ValueError):
        bra.bra_cross_attend(s, q.float(), k, k, None, None, z(2, 5, 64), None, ws)
    with pytest.raises(ValueError):
        bra.bra_cross_attend(s, q, k, k, torch.zeros(2, dtype=torch.int64), None, z(2, 5, 64), None, ws)
    with pytest.raises(ValueError):
        bra.bra_cross_attend(s, q, k[:, :8], k, None, None, z(2, 5, 64), None, ws)
    r = bra.rotary_shape_for(q, None, 2, 0, (0, 8, 8), grid=(1, 5, 1))
    with pytest.raises(ValueError):
        bra.bra_rotary(r, q, None, None, torch.zeros(16), z(2, 5, 64), None)
    with pytest.raises(ValueError):
        bra.bra_rotary(r, q, q, None, torch.zeros(16), z(2, 5, 64), None)
    with pytest.raises(ValueError):
        bra.rotary_shape_for(q, None, 2, 0, (0, 8, 8), grid=(1, 2, 2))
    with pytest.raises(ValueError):
        bra.bra_dropout_add(q, None, 0.1, torch.zeros(2, dtype=torch.int64), z(2, 5, 64))
    with pytest.raises(ValueError):
        bra.bra_dropout_add(q, k, 0.1, torch.zeros(2, dtype=torch.int64), z(2, 5, 64))

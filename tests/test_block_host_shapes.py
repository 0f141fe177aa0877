"""Tensors that are large enough but not laid out as a call reads them: what the
operators' Python layer refuses before it hands pointers on.  The device checks are
replaced, so that all of it runs on CPU tensors; nothing reaches a kernel."""
import contextlib
import warnings

import pytest
import torch

import dynamic_sparse_attention_bra_b200 as bra


@pytest.fixture
def calls(monkeypatch):
    """The C calls that pass the checks, in place of making them."""
    made = []
    monkeypatch.setattr(bra, "_cuda_device", lambda t, where: -1)  # what get_device() says of CPU tensors
    monkeypatch.setattr(bra, "_current_device", lambda: -1)
    monkeypatch.setattr(bra, "_call", lambda where, fn, dev, stream, *args: made.append(where))
    return made


def z(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


# ------------------------------------------------------------------ positions of the rotation

def rotary(calls, B, pos, shape_pos, grid=(1, 2, 3)):
    L = grid[0] * grid[1] * grid[2]
    q = z(B, L, 64)
    s = bra.rotary_shape_for(q, None, 2, 0, (0, 8, 8), grid=grid, pos=shape_pos)
    bra.bra_rotary(s, q, None, pos, torch.zeros(16), z(B, L, 64), None)
    assert calls == ["bra_rotary"]


def positions(*s):
    return z(*s, dtype=torch.int32)


@pytest.mark.parametrize("B,pos,shape_pos", [
    (3, (3, 6, 3), None),        # own positions, a shape that takes them for shared
    (3, (18, 3), None),
    (3, (3, 1, 2, 3, 3), None),
    (3, (3, 9, 3), (3, 9, 3)),   # longer sequences: the entries lie elsewhere
    (2, (4, 6, 3), (1, 6, 3)),
], ids=str)
def test_positions_that_a_shape_would_misread(calls, B, pos, shape_pos):
    with pytest.raises(ValueError, match="pos"):
        rotary(calls, B, positions(*pos), None if shape_pos is None else positions(*shape_pos))
    assert not calls


@pytest.mark.parametrize("B,pos,shape_pos", [
    (3, (3, 6, 3), (3, 6, 3)), (3, (1, 6, 3), (1, 6, 3)), (3, (1, 6, 3), None), (3, (3, 1, 2, 3, 3), (3, 1, 2, 3, 3)),
    (3, (6, 3), None), (1, (6, 3), None), (1, (1, 6, 3), None), (1, (6, 3), (6, 3)), (2, (5, 6, 3), (5, 6, 3)),
    (3, (1, 9, 3), None), (3, (1, 2, 3, 3), None), (3, (18, 3), (18, 3)),
], ids=str)
def test_positions_that_a_shape_reads(calls, B, pos, shape_pos):
    rotary(calls, B, positions(*pos), None if shape_pos is None else positions(*shape_pos))


# --------------------------------------------------- tensors with more in an entry than the shape's

def cross(calls, B=2, Lq=5, Lk=9, backward=True, **other):
    """Both calls on well-formed tensors, but for those named."""
    x = dict(kv_len=z(B, dtype=torch.int32), kv_mask=z(B, Lk, dtype=torch.uint8), o=z(B, Lq, 64),
             lse=z(B, 2, Lq, dtype=torch.float32), grad_o=z(B, Lq, 64), dq=z(B, Lq, 64), dk=z(B, Lk, 64),
             dv=z(B, Lk, 64))
    x.update(other)
    q, k = z(B, Lq, 64), z(B, Lk, 64)
    s = bra.cross_shape_for(q, k, k, 2)
    ws = z(bra.bra_cross_workspace_bytes(s), dtype=torch.uint8)
    bra.bra_cross_attend(s, q, k, k, x["kv_len"], x["kv_mask"], x["o"], x["lse"], ws)
    if backward:
        bra.bra_cross_attend_backward(s, q, k, k, x["kv_len"], x["kv_mask"], x["o"], x["lse"], x["grad_o"], x["dq"],
                                      x["dk"], x["dv"], ws)
    assert calls == ["bra_cross_attend", "bra_cross_attend_backward"][:1 + backward]


@pytest.mark.parametrize("name,shape", [("kv_mask", (2, 12)), ("o", (2, 8, 64)), ("lse", (2, 2, 8)), ("grad_o", (2, 8, 64)),
                                        ("dq", (2, 8, 64)), ("dk", (2, 12, 64)), ("dv", (2, 12, 64)), ("kv_mask", (3, 8)),
                                        ("o", (2, 2, 4, 64))], ids=str)
def test_longer_entries_are_refused(calls, name, shape):
    """A mask of the padded length, an output kept for longer calls: its entries lie elsewhere."""
    t = z(*shape, dtype={"kv_mask": torch.uint8, "lse": torch.float32}.get(name, torch.bfloat16))
    with pytest.raises(ValueError, match=name):
        cross(calls, **{name: t})


def test_longer_heads_of_one_entry_are_refused(calls):
    with pytest.raises(ValueError, match="lse"):
        cross(calls, B=1, lse=z(1, 2, 8, dtype=torch.float32))


@pytest.mark.parametrize("other", [
    dict(o=z(4, 5, 64), lse=z(3, 2, 5, dtype=torch.float32), dq=z(2, 1, 5, 64), dk=z(5, 9, 64)),  # more entries
    dict(o=z(1000), lse=z(100, dtype=torch.float32), kv_mask=z(50, dtype=torch.uint8)),             # flat memory
    dict(kv_len=z(7, dtype=torch.int32), kv_mask=z(2, 3, 3, dtype=torch.bool)),
    dict(B=1, o=z(1, 8, 64), kv_mask=z(1, 12, dtype=torch.uint8), dk=z(1, 12, 64)),                 # one entry's start
    dict(Lq=0, o=z(2, 5, 64), dq=z(2, 0, 64)),
], ids=str)
def test_larger_tensors_that_begin_as_the_shape_says(calls, other):
    cross(calls, **other)


@pytest.mark.parametrize("which", ["residual", "y"])
def test_dropout_refuses_longer_entries(calls, which):
    x, rng = z(2, 5, 64), z(2, dtype=torch.int64)
    t = dict(residual=z(2, 5, 64), y=z(2, 5, 64))
    t[which] = z(2, 8, 64)
    with pytest.raises(ValueError, match=which):
        bra.bra_dropout_add(x, t["residual"], 0.1, rng, t["y"])
    t[which] = z(3, 5, 64)
    bra.bra_dropout_add(x, t["residual"], 0.1, rng, t["y"])
    t[which] = z(1000)
    bra.bra_dropout_add(x, t["residual"], 0.1, rng, t["y"])
    assert calls == ["bra_dropout_add"] * 2


# ------------------------------------------------------------------ the workspace's device

def test_the_workspace_s_size_is_that_of_the_tensors_device(monkeypatch):
    """Device 1, with more SMs than the current device 0, splits further and needs more."""
    current, made = [0], []

    @contextlib.contextmanager
    def device(i):
        current.append(i)
        yield
        current.pop()
    monkeypatch.setattr(bra, "_current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(bra, "_cuda_device", lambda t, where: 1)
    monkeypatch.setattr(bra, "_same_tokens", lambda *a: None)
    monkeypatch.setattr(bra, "_dense", lambda t, name, dtype, numel, dev: not made.append((name, numel)))
    monkeypatch.setattr(bra, "bra_cross_workspace_bytes", lambda s: 1000 + 1000 * current[-1])
    monkeypatch.setattr(bra, "_call", lambda *a: None)
    q, k = z(2, 5, 64), z(2, 9, 64)
    s = bra.cross_shape_for(q, k, k, 2)
    bra.bra_cross_attend(s, q, k, k, None, None, q, None, q)
    bra.bra_cross_attend_backward(s, q, k, k, None, None, q, q, q, q, k, k, q)
    assert [n for name, n in made if name == "workspace"] == [2000, 2000]
    sizes = []
    monkeypatch.setattr(torch, "zeros", lambda n, **kw: sizes.append(n) or q)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    bra.cross_attention(q, k, k, 2)
    assert sizes == [2000] and current == [0]


# ------------------------------------------------------------------ scales

@pytest.mark.parametrize("scale,code", [(2.4e38, bra.BRA_ERR_INVALID_ARG), (3.4e38, bra.BRA_ERR_INVALID_ARG),
                                        (1.7e38, bra.BRA_OK), (1e-45, bra.BRA_OK)])
def test_scales_whose_powers_of_two_overflow(scale, code):
    """The kernels multiply by scale log2(e), which has to be finite too."""
    q = z(0, 5, 64)
    s = bra.cross_shape_for(q, q, q, 2, scale=scale)
    p = 1 << 20  # never followed: there is no entry
    assert bra._lib.bra_cross_attend(s, *([p] * 8), None) == code
    assert (bra.bra_cross_workspace_bytes(s) == 0) == (code != bra.BRA_OK)


# ------------------------------------------------------------------ gradients that the wrapper does not give

def test_the_wrapper_says_that_it_gives_no_gradients(calls, monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    q, k = z(2, 5, 64), z(2, 9, 64)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        bra.cross_attention(q, k, k, 2)
        with torch.no_grad():
            bra.cross_attention(q.requires_grad_(), k, k, 2)
    for args in ((q, k, k), (q.detach(), k.requires_grad_(), k), (q.detach(), k.detach(), k)):
        with pytest.warns(UserWarning, match="bra_cross_attend_backward"):
            o, lse = bra.cross_attention(*args, 2)
        assert not o.requires_grad
    assert len(calls) == 5

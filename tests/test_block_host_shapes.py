"""Tensors that are large enough but not laid out as a call reads them: what the
operators' Python layer refuses before it hands pointers on.  The device checks are
replaced, so that all of it runs on CPU tensors; nothing reaches a kernel."""
import contextlib

import pytest
import torch

import dynamic_sparse_attention_bra_b200 as bra


@pytest.fixture
def calls(monkeypatch):
    """The C calls that pass the checks, in place of making them."""
    made = []
    monkeypatch.setattr(bra, "_cuda_device", lambda t, where: -1)  # what get_device() says of CPU tensors
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
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

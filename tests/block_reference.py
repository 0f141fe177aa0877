"""64-bit definitions of the conditioned block's operators, written from their
formulas with elementary torch operations: what the GPU tests compare with,
and what the CPU tests pin by differences, closed forms and published values."""
from __future__ import annotations

import math

import torch

BF16_STEP = torch.finfo(torch.bfloat16).eps / 2  # half a step, relative
F32_STEP = torch.finfo(torch.float32).eps / 2


def step(dtype) -> float:
    return BF16_STEP if dtype == torch.bfloat16 else F32_STEP


def valid_states(B, Lk, kv_len=None, kv_mask=None, device="cpu"):
    ok = torch.ones((B, Lk), dtype=torch.bool, device=device)
    if kv_len is not None:
        ok &= torch.arange(Lk, device=device)[None] < kv_len.to(device)[:, None]
    if kv_mask is not None:
        ok &= kv_mask.to(device).bool()
    return ok


def _heads(x, n):
    B, L, C = x.shape
    return x.double().reshape(B, L, n, C // n).transpose(1, 2)  # [B, n, L, d]


def cross(q, k, v, heads, kv_heads, ok, scale=None, grad=None):
    """A dict of 64-bit o, lse, p (and dq, dk, dv, ds) and of the sums that bound rounding errors."""
    B, Lq, C = q.shape
    d, rep = C // heads, heads // kv_heads
    scale = d ** -0.5 if scale is None else scale
    zero = ~ok[:, None, :, None]
    Q = _heads(q, heads)
    K = _heads(k, kv_heads).masked_fill(zero, 0.0).repeat_interleave(rep, 1)  # what is masked is never used
    V = _heads(v, kv_heads).masked_fill(zero, 0.0).repeat_interleave(rep, 1)
    s = (Q @ K.transpose(2, 3)) * scale
    s = s.masked_fill(~ok[:, None, None], -math.inf)
    some = ok.any(1)[:, None, None, None]
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:3], -math.inf, dtype=torch.float64,
                                                               device=q.device)
    p = torch.where(some, torch.exp(s - torch.where(some[..., 0], lse, 0.0)[..., None]), 0.0)
    back = lambda x: x.transpose(1, 2).reshape(B, x.shape[2], -1)
    join = lambda x: back(x.reshape(B, kv_heads, rep, *x.shape[2:]).sum(2))
    o = p @ V
    r = {"o": back(o), "lse": lse, "p": p, "abs_o": back(p @ V.abs()),
         "smax": float((Q.abs() @ K.abs().transpose(2, 3)).max()) * scale if s.numel() else 0.0}
    if grad is not None:
        G = _heads(grad, heads)
        dp = G @ V.transpose(2, 3)
        D = (p * dp).sum(-1, keepdim=True)
        ds = p * (dp - D)
        r.update(dq=back(ds @ K) * scale, dk=join(ds.transpose(2, 3) @ Q) * scale, dv=join(p.transpose(2, 3) @ G))
        r["abs_dq"] = back(ds.abs() @ K.abs()) * scale
        r["abs_dk"] = join(ds.abs().transpose(2, 3) @ Q.abs()) * scale
        r["abs_dv"] = join(p.transpose(2, 3) @ G.abs())
        # for fp32 terms: everything in absolute values, nothing cancelled
        big = p * (G.abs() @ V.abs().transpose(2, 3) + (p * (G.abs() @ V.abs().transpose(2, 3))).sum(-1, keepdim=True))
        r["all_dq"] = back(big @ K.abs()) * scale
        r["all_dk"] = join(big.transpose(2, 3) @ Q.abs()) * scale
        # |D - D0|, D0 of a rounded O, times sum_j P_j |k_j|
        D0 = (G.abs() * o.abs()).sum(-1, keepdim=True)
        r["rest_dq"] = back(D0 * (p @ K.abs())) * scale
    return r


def cross_bounds(r, dtype, d, Lk, rows):
    """Error bounds of each output, from the roundings that the kernels make.

    bf16: P and dS enter a product rounded once (u = half a bf16 step), and
    each output is rounded once.  The correction of D multiplies a sum of
    rounded P by |D - D0| <= u sum |dO||O|, which adds u^2.  fp32 terms: a
    score is a sum of d products (d + 2 roundings of sums that are at most
    smax), it changes P by as much; the sums over n terms n roundings; the
    exponential 2^-21 (its argument's rounding included)."""
    u = step(dtype)
    half = u if dtype == torch.bfloat16 else 0.0
    e = 4 * F32_STEP * ((d + 4) * (r["smax"] + 1) + Lk + rows + d) + 2.0 ** -20
    b = {"o": (half + e) * r["abs_o"] + u * r["o"].abs() + 1e-30,
         "lse": torch.full_like(r["lse"], e) + 2 * F32_STEP * torch.where(torch.isfinite(r["lse"]), r["lse"].abs(), 0.0)}
    if "dq" in r:
        tiny = 2.0 ** -126
        b["dq"] = half * r["abs_dq"] + half * half * r["rest_dq"] + e * r["all_dq"] + u * r["dq"].abs() + tiny
        b["dk"] = half * r["abs_dk"] + e * r["all_dk"] + u * r["dk"].abs() + tiny
        b["dv"] = (half + e) * r["abs_dv"] + u * r["dv"].abs() + tiny
        if dtype == torch.bfloat16:  # a product of two roundings
            for x in ("dq", "dk", "dv"):
                b[x] = b[x] * (1 + 2 * u)
    return b


def rotary(x, heads, pairs, inv_freq, pos, interleaved=False, inverse=False):
    """pos int [B or 1, L, 3]; 64 bits throughout."""
    B, L, C = x.shape
    d, P = C // heads, sum(pairs)
    axis = torch.tensor([0] * pairs[0] + [1] * pairs[1] + [2] * pairs[2], device=x.device)
    a = pos[:, :, axis].double() * inv_freq.double()
    c, s = torch.cos(a)[:, :, None], torch.sin(a)[:, :, None] * (-1 if inverse else 1)
    y = x.double().reshape(B, L, heads, d).clone()
    z = y.clone()
    i1 = torch.arange(P, device=x.device) * (2 if interleaved else 1)
    i2 = i1 + (1 if interleaved else P)
    z[..., i1] = y[..., i1] * c - y[..., i2] * s
    z[..., i2] = y[..., i2] * c + y[..., i1] * s
    return z.reshape(B, L, C)


def grid_positions(T, H, W, device="cpu"):
    t, y, x = torch.meshgrid(torch.arange(T), torch.arange(H), torch.arange(W), indexing="ij")
    return torch.stack((t, y, x), -1).reshape(1, T * H * W, 3).to(torch.int32).to(device)


def philox4x32(key: int, counter: int) -> list[int]:
    """Ten rounds of Philox4x32 in Python integers; ``counter`` has 128 bits, ``key`` 64."""
    x = [(counter >> (32 * i)) & 0xFFFFFFFF for i in range(4)]
    k = [key & 0xFFFFFFFF, key >> 32 & 0xFFFFFFFF]
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(b >> 32) ^ x[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ x[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def keeps(n: int, unit: int, p: float, seed: int, offset: int) -> torch.Tensor:
    """The mask of n elements, element by element."""
    units = -(-n // unit)
    words = []
    for c in range(-(-units // 4)):
        words += philox4x32(seed, (offset + c) & (2 ** 64 - 1))
    on = torch.tensor([w >= p * 2.0 ** 32 for w in words[:units]], dtype=torch.bool)
    return on.repeat_interleave(unit)[:n]

"""How far the bf16 results of cross attention may be from 64 bits in the norm.

The kernels round P and dS once to bf16 as operands and every result once; everything
else is fp32.  A rounding to nearest is off by at most 2^-8 of the value's power of two,
evenly spread, so that its mean square is at most (2^-8)^2 / 3 of the value's square;
the roundings are independent, and the mean squares of a sum's errors add up:

    O   sum_j P_j^2 v_j^2                                      + O^2
    dQ  scale^2 sum_j dS_j^2 (k_j - kbar)^2 + (D - D0)^2 terms + dQ^2
    dK  scale^2 sum_r (dS_r^2 + P_r^2 sum_j dS_rj^2) q_r^2     + dK^2
    dV  sum_r P_r^2 dO_r^2                                     + dV^2

times (2^-8)^2 / 3.  kbar = sum_j P_j k_j: the sum of the rounded dS times it is taken
out of dQ, and with it what the roundings have in common; the same sum corrects D, whose
error then is that of the roundings (dK's second term).  An error in D that is left in
dQ, or P with fewer bits, multiplies these norms; bounds that add every rounding at its
worst (block_reference.cross_bounds) let both pass."""
from __future__ import annotations

import torch

from block_reference import _heads

MEAN_SQUARE = (2.0 ** -8) ** 2 / 3
# the values' own powers of two leave the true mean square at 0.54 of MEAN_SQUARE; sums of a few
# thousand squares stray by some hundredths
SLACK = 1.1


def error_norms(q, k, v, heads, kv_heads, ok, r, grad, scale=None):
    """The expected norms of o's, dq's, dk's and dv's errors; r as block_reference.cross gives it."""
    B, Lq, C = q.shape
    d, rep = C // heads, heads // kv_heads
    scale = d ** -0.5 if scale is None else scale
    zero = ~ok[:, None, :, None]
    Q, G = _heads(q, heads), _heads(grad, heads)
    K = _heads(k, kv_heads).masked_fill(zero, 0.0).repeat_interleave(rep, 1)
    V = _heads(v, kv_heads).masked_fill(zero, 0.0).repeat_interleave(rep, 1)
    p, o = r["p"], r["p"] @ V
    dp = G @ V.transpose(2, 3)
    ds2 = (p * (dp - (p * dp).sum(-1, keepdim=True))).square()
    p2, kbar = p.square(), p @ K
    rows = ds2.sum(-1, keepdim=True)
    d0 = (G * o).square().sum(-1, keepdim=True) * MEAN_SQUARE  # (D - D0)^2, D0 of a rounded O
    var = {"o": (p2 @ V.square()).sum() + r["o"].square().sum()}
    spread = ds2 @ K.square() - 2 * (ds2 @ K) * kbar + rows * kbar.square()
    var["dq"] = scale ** 2 * (spread + d0 * (p2 @ (K.square()))
                              + d0 * (p2 @ K.square() + p2.sum(-1, keepdim=True) * kbar.square())).sum()
    var["dq"] = var["dq"] + r["dq"].square().sum()
    var["dk"] = scale ** 2 * ((ds2 + p2 * rows).transpose(2, 3) @ Q.square()).sum() + r["dk"].square().sum()
    var["dv"] = (p2.transpose(2, 3) @ G.square()).sum() + r["dv"].square().sum()
    return {x: float(s * MEAN_SQUARE) ** 0.5 for x, s in var.items()}


def limits(norms, r):
    """What a result's error norm may be: the roundings', and 2^-18 of its sums in absolute values for fp32."""
    whole = {"o": "abs_o", "dq": "all_dq", "dk": "all_dk", "dv": "abs_dv"}
    return {x: SLACK * n + 2.0 ** -18 * float(r[whole[x]].norm()) for x, n in norms.items()}

"""Measured cases of the conditioned block's operators: cross attention to an encoder's states,
rotary positions with several axes, and dropout with the residual's sum.

``run`` computes them in their plain form (elementary torch operations in 32 bits, rounded once)
or, where ``own`` is true, through the framework's entry points; ``exact`` computes the
definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}

# A cross-attention case: B entries of Lq query tokens and Lk states, heads query heads of size d over
# kv_heads state heads; valid: "all", "len" (a length for each entry, one entry empty, one full) or
# "mask" (a truth value for each state). train: gradients too.
# A rotary case: a grid of T x H x W tokens for each of B entries ("grid") or L tokens with given
# positions ("given"); pt, ph, pw rotation pairs of time, height and width.
# A dropout case: B entries of L tokens of C channels; unit: elements that share a draw.


def _cross(name, B, Lq, Lk, heads, kv_heads, d, dtype, valid="all", train=False):
    return dict(name=name, op="cross", B=B, Lq=Lq, Lk=Lk, heads=heads, kv_heads=kv_heads, d=d, dtype=dtype,
                valid=valid, train=train)


def _rotary(name, B, T, H, W, heads, kv_heads, d, pt, ph, pw, dtype, positions="grid", interleaved=False,
            inverse=False):
    return dict(name=name, op="rotary", B=B, T=T, H=H, W=W, heads=heads, kv_heads=kv_heads, d=d, pt=pt, ph=ph, pw=pw,
                dtype=dtype, positions=positions, interleaved=interleaved, inverse=inverse)


def _dropout(name, B, L, C, unit, p, dtype, residual=True):
    return dict(name=name, op="dropout", B=B, L=L, C=C, unit=unit, p=p, dtype=dtype, residual=residual)


def listed():
    return [
        # one query token of one image, 49 states (a 7 x 7 map): latency
        _cross("token_short", 1, 1, 49, 2, 2, 32, "bf16"),
        # a decoder's next token for 16 entries over long states with grouped heads: the bytes of K and V
        _cross("token_long", 16, 1, 16384, 32, 8, 64, "bf16", "len"),
        # the stage-1 map's tokens reading padded text-like states
        _cross("map_to_short_states", 64, 3136, 77, 2, 2, 32, "bf16", "len"),
        # the high-resolution map reading a 64 x 64 map's tokens
        _cross("highres_to_map", 2, 16384, 4096, 2, 2, 32, "bf16"),
        # wide heads, grouped: a decoder's prompt over an encoder's output
        _cross("prompt_grouped", 4, 2048, 2048, 16, 4, 128, "bf16", "len"),
        # full precision, an odd number of states with a mask
        _cross("map_f32", 8, 784, 333, 4, 4, 32, "f32", "mask"),
        # a training step on the stage-2 map, 14 x 14 states
        _cross("train_stage2", 64, 784, 196, 4, 4, 32, "bf16", "mask", True),
        # a training step over long states, grouped heads
        _cross("train_long", 2, 4096, 4096, 8, 2, 64, "bf16", "len", True),
        # rotary positions (height, width) of the stage-1 map's Q and K
        _rotary("rotary_map", 64, 1, 56, 56, 2, 2, 32, 0, 8, 8, "bf16"),
        # video tokens with given positions in full precision, the inverse rotation (gradients)
        _rotary("rotary_video_back", 2, 12, 24, 23, 8, 2, 64, 8, 12, 12, "f32", "given", True, True),
        # dropout and residual after the stage-1 attention
        _dropout("dropout_stage1", 64, 3136, 64, 1, 0.1, "bf16"),
        # stochastic depth for each sample, full precision, stage 3
        _dropout("depth_stage3", 64, 196, 256, 196 * 256, 0.2, "f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["token", "map", "map", "train", "train", "rotary", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("token", "map", "train"):
        d = rng.choice([32, 32, 64, 128])
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4])
        valid = rng.choice(["all", "len", "mask"])
        B = _log(rng, 1, 64)
        if kind == "token":
            Lq, Lk = rng.choice([1, 1, 2, 3, 5, 8]), _log(rng, 1, 32768)
            while B * Lk * kv * d * ELEM[dtype] > 1 << 28:  # K and V each at most 268 MB
                B, Lk = max(1, B // 2), max(1, Lk * 3 // 4)
        else:
            Lq, Lk = _log(rng, 9, 16384), _log(rng, 16 if kind == "train" else 1, 8192)
            most = (1 << 31 if kind == "map" else 1 << 32) // (1 if dtype == "bf16" else 4)
            while B * heads * Lq * Lk * d > most:  # products of Q and K
                B, Lq = max(1, B * 2 // 3), max(9, Lq * 3 // 4)
        case = _cross("", B, Lq, Lk, heads, kv, d, dtype, valid, kind == "train")
    elif kind == "rotary":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4])
        d = rng.choice([32, 32, 64, 128])
        half = d // 2
        pt = rng.choice([0, half // 4, half // 2 - 3])
        ph = (half - pt) // 2
        pw = ph if rng.random() < 0.5 else half - pt - ph  # the first leaves channels that do not turn
        T, H, W = rng.choice([1, 1, 5, 16]), _log(rng, 1, 128), _log(rng, 1, 128)
        B = _log(rng, 1, 64)
        while B * T * H * W * (heads + kv) * d > 1 << 26:
            B, H = max(1, B // 2), max(1, H * 3 // 4)
        case = _rotary("", B, T, H, W, heads, kv, d, pt, ph, pw, dtype, rng.choice(["grid", "given"]),
                       rng.random() < 0.5, rng.random() < 0.5)
    else:
        B, L, C = _log(rng, 1, 64), _log(rng, 1, 16384), 32 * rng.choice([1, 2, 3, 4, 8, 16])
        while B * L * C > 1 << 24:
            B, L = max(1, B // 2), max(1, L * 3 // 4)
        case = _dropout("", B, L, C, rng.choice([1, 1, C, L * C]), rng.choice([0.05, 0.1, 0.25, 0.5]), dtype,
                        rng.random() < 0.6)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 16 + stream)
    return g


def _normal(seed, stream, shape, dtype, mean=0.0):
    """Tokens around a mean for each entry and channel, as projected feature maps are."""
    g = _gen(seed, stream)
    x = torch.randn(shape, generator=g, device="cuda")
    mu = torch.randn((shape[0], 1, shape[-1]), generator=g, device="cuda")
    return x.add_(mu, alpha=0.5).add_(mean).to(dtype)


def _valid(c, seed):
    """(lengths int32 [B] or None, mask uint8 [B, Lk] or None)."""
    B, Lk = c["B"], c["Lk"]
    if c["valid"] == "len":
        n = torch.randint(Lk - Lk // 2, Lk + 1, (B,), generator=_gen(seed, 9), device="cuda", dtype=torch.int32)
        if B >= 4:
            n[1], n[2] = 0, Lk
        return n, None
    if c["valid"] == "mask":
        return None, (torch.rand((B, Lk), generator=_gen(seed, 9), device="cuda") < 0.75).to(torch.uint8)
    return None, None


def _inv_freq(c):
    """One frequency for each pair, falling from 1 along each axis."""
    f = [10000.0 ** (-i / n) for n in (c["pt"], c["ph"], c["pw"]) for i in range(n)]
    return torch.tensor(f, dtype=torch.float32, device="cuda")


def prepare(case, seed):
    c, t = case, DTYPES[case["dtype"]]
    s = {"case": dict(c)}
    if c["op"] == "cross":
        B, Lq, Lk, d = c["B"], c["Lq"], c["Lk"], c["d"]
        s["q"] = _normal(seed, 0, (B, Lq, c["heads"] * d), t)
        s["k"] = _normal(seed, 1, (B, Lk, c["kv_heads"] * d), t)
        s["v"] = _normal(seed, 2, (B, Lk, c["kv_heads"] * d), t)
        s["n"], s["mask"] = _valid(c, seed)
        if c["train"]:
            s["do"] = _normal(seed, 3, (B, Lq, c["heads"] * d), t)
    elif c["op"] == "rotary":
        B, L = c["B"], c["T"] * c["H"] * c["W"]
        s["q"] = _normal(seed, 0, (B, L, c["heads"] * c["d"]), t)
        s["k"] = _normal(seed, 1, (B, L, c["kv_heads"] * c["d"]), t)
        s["inv_freq"] = _inv_freq(c)
        s["pos"] = None
        if c["positions"] == "given":  # clips that start anywhere in a long video
            grid = torch.stack(_grid(c), -1)
            start = torch.randint(0, 100000, (B, 1, 3), generator=_gen(seed, 4), device="cuda")
            s["pos"] = (grid[None] + start).to(torch.int32).contiguous()
    else:
        shape = (c["B"], c["L"], c["C"])
        s["x"] = _normal(seed, 0, shape, t)
        s["residual"] = _normal(seed, 1, shape, t) if c["residual"] else None
        s["rng"] = torch.tensor([seed * 0x9E3779B97F4A7C15 % (1 << 63), 1000003 * seed], dtype=torch.int64,
                                device="cuda")
    if own:  # the plan, the workspace and the outputs' memory, which a program keeps
        import dynamic_sparse_attention_bra_b200 as bra
        if c["op"] == "cross":
            s["shape"] = bra.cross_shape_for(s["q"], s["k"], s["v"], c["heads"], c["kv_heads"])
            s["ws"] = torch.zeros(bra.bra_cross_workspace_bytes(s["shape"]), dtype=torch.uint8, device="cuda")
            s["out"] = [torch.empty_like(s["q"])]
            s["lse"] = None
            if c["train"]:
                s["lse"] = torch.empty((c["B"], c["heads"], c["Lq"]), dtype=torch.float32, device="cuda")
                s["out"] += [torch.empty_like(s[x]) for x in "qkv"]
        elif c["op"] == "rotary":
            s["out"] = [torch.empty_like(s["q"]), torch.empty_like(s["k"])]
            s["shape"] = bra.rotary_shape_for(s["q"], s["k"], c["heads"], c["kv_heads"], (c["pt"], c["ph"], c["pw"]),
                                              grid=(c["T"], c["H"], c["W"]), pos=s["pos"],
                                              interleaved=c["interleaved"], inverse=c["inverse"])
        else:
            s["out"] = [torch.empty_like(s["x"])]
    return s


# -------------------------------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return {"cross": _plain_cross, "rotary": _plain_rotary, "dropout": _plain_dropout}[c["op"]](s, c)


def _run_own(s, c):
    import dynamic_sparse_attention_bra_b200 as bra
    if c["op"] == "cross":
        o = s["out"][0]
        bra.bra_cross_attend(s["shape"], s["q"], s["k"], s["v"], s["n"], s["mask"], o, s["lse"], s["ws"])
        if not c["train"]:
            return o
        dq, dk, dv = s["out"][1:]
        bra.bra_cross_attend_backward(s["shape"], s["q"], s["k"], s["v"], s["n"], s["mask"], o, s["lse"], s["do"], dq,
                                      dk, dv, s["ws"])
        return o, s["lse"], dq, dk, dv
    if c["op"] == "rotary":
        q, k = s["out"]
        bra.bra_rotary(s["shape"], s["q"], s["k"], s["pos"], s["inv_freq"], q, k)
        return q, k
    bra.bra_dropout_add(s["x"], s["residual"], c["p"], s["rng"], s["out"][0], unit=c["unit"])
    return s["out"][0]


def _plain_cross(s, c):
    B, Lq, Lk, hk, d = c["B"], c["Lq"], c["Lk"], c["kv_heads"], c["d"]
    rep, t = c["heads"] // hk, s["q"].dtype
    # [B, state heads, group's heads x tokens, d]
    q = s["q"].float().view(B, Lq, hk, rep, d).permute(0, 2, 3, 1, 4).reshape(B, hk, rep * Lq, d)
    k = s["k"].float().view(B, Lk, hk, d).transpose(1, 2)
    v = s["v"].float().view(B, Lk, hk, d).transpose(1, 2)
    sc = torch.matmul(q * d ** -0.5, k.transpose(2, 3))
    bad = None
    if s["n"] is not None:
        bad = torch.arange(Lk, device=q.device)[None] >= s["n"][:, None]
    elif s["mask"] is not None:
        bad = s["mask"] == 0
    if bad is not None:
        sc.masked_fill_(bad[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    if bad is not None:
        m = m.masked_fill(m == -math.inf, 0.0)
    p = sc.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.mul_(torch.where(total > 0, 1.0 / total, 0.0))
    o = torch.matmul(p, v)

    def rows(x, like):
        return x.view(B, hk, rep, Lq, d).permute(0, 3, 1, 2, 4).reshape(B, Lq, -1).to(like)

    if not c["train"]:
        return rows(o, t)
    lse = (m + total.log()).view(B, hk, rep, Lq).reshape(B, c["heads"], Lq)
    do = s["do"].float().view(B, Lq, hk, rep, d).permute(0, 2, 3, 1, 4).reshape(B, hk, rep * Lq, d)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(d ** -0.5)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)

    def states(x):
        return x.transpose(1, 2).reshape(B, Lk, hk * d).to(t)

    return rows(o, t), lse, rows(dq, t), states(dk), states(dv)


def _grid(c):
    """Time, height and width of each of the T x H x W tokens."""
    i = torch.arange(c["T"] * c["H"] * c["W"], device="cuda")
    return i // (c["H"] * c["W"]), i // c["W"] % c["H"], i % c["W"]


def _angles(s, c):
    """[1 or B, L, pairs] in 64 bits: far positions lose their angle in 32."""
    pos = torch.stack(_grid(c), -1)[None] if s["pos"] is None else s["pos"]
    axis = torch.tensor([0] * c["pt"] + [1] * c["ph"] + [2] * c["pw"], device="cuda")
    return pos[:, :, axis].double() * s["inv_freq"].double()


def _plain_rotary(s, c):
    a = _angles(s, c)
    cos, sin = a.cos().float()[:, :, None], a.sin().float()[:, :, None]
    if c["inverse"]:
        sin = -sin
    P = cos.shape[-1]

    def turn(x, heads):
        B, L, C = x.shape
        y = x.float().view(B, L, heads, c["d"])
        if c["interleaved"]:
            x1, x2 = y[..., 0:2 * P:2], y[..., 1:2 * P:2]
            z = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
        else:
            x1, x2 = y[..., :P], y[..., P:2 * P]
            z = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
        return torch.cat((z, y[..., 2 * P:]), -1).view(B, L, C).to(x.dtype)

    return turn(s["q"], c["heads"]), turn(s["k"], c["kv_heads"])


M0, M1, W0, W1, LOW = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF


def _philox(seed, first, count):
    """Words of Philox4x32-10 (Salmon and others, 2011) for ``count`` counters from ``first``: int64 [count, 4]."""
    ctr = first + torch.arange(count, device="cuda")
    x = [ctr & LOW, (ctr >> 32) & LOW, torch.zeros_like(ctr), torch.zeros_like(ctr)]
    k0, k1 = seed & LOW, (seed >> 32) & LOW
    for _ in range(10):
        a, b = x[0] * M0, x[2] * M1  # 64-bit products; the high half survives the wrap of the sign
        x = [((b >> 32) & LOW) ^ x[1] ^ k0, b & LOW, ((a >> 32) & LOW) ^ x[3] ^ k1, a & LOW]
        k0, k1 = (k0 + W0) & LOW, (k1 + W1) & LOW
    return torch.stack(x, -1)


def _keep(s, c):
    n = c["B"] * c["L"] * c["C"]
    units = -(-n // c["unit"])
    w = _philox(s["rng"][0], s["rng"][1], -(-units // 4)).flatten()[:units] >= math.ceil(c["p"] * 2 ** 32)
    if c["unit"] > 1:
        w = w[:, None].expand(-1, c["unit"]).reshape(-1)[:n]
    return w.view(c["B"], c["L"], c["C"])


def _plain_dropout(s, c):
    y = torch.where(_keep(s, c), s["x"].float() * (1.0 / (1.0 - c["p"])), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


# -------------------------------------------------------------------------- cost and 64-bit values

def work(case):
    c, e = case, ELEM[case["dtype"]]
    if c["op"] == "cross":
        part = 1.0 if c["valid"] == "all" else 0.75  # of the states
        q = c["B"] * c["Lq"] * c["heads"] * c["d"]
        kv = 2 * c["B"] * c["Lk"] * c["kv_heads"] * c["d"] * part
        pairs = q * c["Lk"] * part
        rows = c["B"] * c["Lq"] * c["heads"]
        if not c["train"]:
            return {"bytes": e * (2 * q + kv), "flops": 4 * pairs}
        # forward: Q, K, V in, O and the log sums out; backward: Q, K, V, O, dO, log sums in, the gradients out
        grads = 2 * c["B"] * c["Lk"] * c["kv_heads"] * c["d"]
        return {"bytes": e * (2 * q + kv) + e * (4 * q + kv + grads) + 8 * rows, "flops": 14 * pairs}
    if c["op"] == "rotary":
        tokens = c["B"] * c["T"] * c["H"] * c["W"]
        n = tokens * (c["heads"] + c["kv_heads"]) * c["d"]
        return {"bytes": 2 * e * n + (12 * tokens if c["positions"] == "given" else 0), "flops": 3 * n}
    n = c["B"] * c["L"] * c["C"]
    return {"bytes": e * n * (3 if c["residual"] else 2), "flops": 2 * n}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"cross": _exact_cross, "rotary": _exact_rotary, "dropout": _exact_dropout}[case["op"]](s, case)


def _exact_cross(s, c):
    B, Lq, Lk, d, h = c["B"], c["Lq"], c["Lk"], c["d"], c["heads"]
    rep = h // c["kv_heads"]
    o = torch.zeros((B, Lq, h, d), dtype=torch.float64, device="cuda")
    dq, lse = torch.zeros_like(o), torch.full((B, h, Lq), -math.inf, dtype=torch.float64, device="cuda")
    dk = torch.zeros((B, Lk, c["kv_heads"], d), dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    for b in range(B):
        if s["n"] is not None:
            at = torch.arange(int(s["n"][b]), device="cuda")
        elif s["mask"] is not None:
            at = s["mask"][b].nonzero()[:, 0]
        else:
            at = torch.arange(Lk, device="cuda")
        if not len(at):
            continue
        for j in range(c["kv_heads"]):
            k = s["k"][b, at, j * d:(j + 1) * d].double()
            v = s["v"][b, at, j * d:(j + 1) * d].double()
            gk, gv = torch.zeros_like(k), torch.zeros_like(v)
            for i in range(j * rep, (j + 1) * rep):
                q = s["q"][b, :, i * d:(i + 1) * d].double()
                z = q @ k.T / math.sqrt(d)
                lse[b, i] = torch.logsumexp(z, 1)
                p = torch.exp(z - lse[b, i][:, None])
                o[b, :, i] = p @ v
                if c["train"]:
                    g = s["do"][b, :, i * d:(i + 1) * d].double()
                    dp = g @ v.T
                    dz = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[b, :, i] = dz @ k
                    gk += dz.T @ q
                    gv += p.T @ g
            dk[b, at, j], dv[b, at, j] = gk, gv
    if not c["train"]:
        return o.view(B, Lq, -1)
    return o.view(B, Lq, -1), lse, dq.view(B, Lq, -1), dk.view(B, Lk, -1), dv.view(B, Lk, -1)


def _exact_rotary(s, c):
    a = _angles(s, c) * (-1 if c["inverse"] else 1)
    w = torch.polar(torch.ones_like(a), a)[:, :, None]
    P = w.shape[-1]

    def turn(x, heads):
        B, L, C = x.shape
        y = x.double().view(B, L, heads, c["d"]).clone()
        one, two = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if c["interleaved"] else (slice(0, P), slice(P, 2 * P))
        z = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * w
        y[..., one], y[..., two] = z.real, z.imag
        return y.view(B, L, C)

    return turn(s["q"], c["heads"]), turn(s["k"], c["kv_heads"])


def _exact_dropout(s, c):
    n, x = c["B"] * c["L"] * c["C"], s["x"].double().flatten()
    word = torch.arange(n, device="cuda") // c["unit"]
    seed, first = (int(v) for v in s["rng"].tolist())
    words = _philox(torch.tensor(seed, device="cuda"), first, int(word[-1]) // 4 + 1)
    y = x * (words[word // 4, word % 4] >= c["p"] * 2.0 ** 32) / (1 - c["p"])
    if s["residual"] is not None:
        y = y + s["residual"].double().flatten()
    return y.view(c["B"], c["L"], c["C"])

"""The mbarrier protocols of the tcgen05 cross-attention kernels, as roles run over
random interleavings by the model of test_protocol_model.py (a wait that could pass
before its phase's predecessor has completed is EARLY, one that could sleep past its
phase ALIAS, roles that cannot move a DEADLOCK).

Forward: two issuing warps (even and odd tiles), the loader, the warp that passes
landed blocks on, and each tile's softmax.  Backward: the issuer of S and dP, that of
the sums, the loader, the passing warp, and the groups of row threads.  A role's
threads are one role; their arrivals are one arrival.  Units of no block, of one, and
of several; tiles without rows; masked units, whose softmax also waits for the block.
A negative case is the form of the backward that failed on a GPU: its row threads
waited for the last block's buffer instead of a barrier of the units."""
import pytest

from test_protocol_model import Bar, ProtocolError, run


def forward(units, tiles, ring, bufs, alias):
    """units: (blocks, tiles with rows, masked)."""
    bars = {f"drain{w}": Bar("drain", 1) for w in range(2)}
    for s in range(ring):
        bars[f"land{s}"], bars[f"full{s}"] = Bar(f"land{s}"), Bar(f"full{s}")
        bars[f"empty{s}"] = Bar(f"empty{s}", tiles)
    for t in range(tiles):
        for x in range(2):
            for n in ("qf", "qe", "sf", "sr", "pf", "od"):
                bars[f"{n}{t}{x}"] = Bar(f"{n}{t}{x}")

    def issuer(w):
        own = list(range(w, tiles, 2))
        i, done, use = 0, {t: 0 for t in own}, {t: 0 for t in own}

        def qk(t, b, nb):
            at, c = i + b, done[t] + b
            yield ("wait", f"full{at % ring}", at // ring)
            if c >= bufs:
                yield ("wait", f"{'od' if alias else 'sr'}{t}{c % bufs}", c // bufs - 1)
            yield ("arrive", f"sf{t}{c % bufs}")
            if b == nb - 1:
                yield ("arrive", f"qe{t}{use[t] & 1}")

        def pv(t, b):
            at, c = i + b, done[t] + b
            yield ("wait", f"pf{t}{c % bufs}", c // bufs)
            yield ("arrive", f"od{t}{c % bufs}")
            yield ("arrive", f"empty{at % ring}")

        for nb, rows, _ in units:
            for b in range(-1, nb):
                for t in own:
                    if t < rows and b + 1 < nb:
                        if b < 0:
                            yield ("wait", f"qf{t}{use[t] & 1}", use[t] >> 1)
                        yield from qk(t, b + 1, nb)
                if b < 0:
                    continue
                for t in own:
                    if t < rows:
                        yield from pv(t, b)
                    else:
                        yield ("wait", f"full{(i + b) % ring}", (i + b) // ring)
                        yield ("arrive", f"empty{(i + b) % ring}")
            i += nb
            for t in own:
                if t < rows and nb:
                    done[t] += nb
                    use[t] += 1

    def loader():
        i, uses = 0, [0] * tiles
        for nb, rows, _ in units:
            if not nb:
                continue
            for t in range(rows):
                u = uses[t]
                uses[t] += 1
                if u >= 2:
                    yield ("wait", f"qe{t}{u & 1}", (u >> 1) - 1)
                yield ("arrive", f"qf{t}{u & 1}")
            for _ in range(nb):
                if i >= ring:
                    yield ("wait", f"empty{i % ring}", i // ring - 1)
                yield ("arrive", f"land{i % ring}")
                i += 1

    def passing():
        for i in range(sum(u[0] for u in units)):
            yield ("wait", f"land{i % ring}", i // ring)
            yield ("arrive", f"full{i % ring}")

    def softmax(t):
        i = done = 0
        for nb, rows, masked in units:
            if t >= rows:
                i += nb
                continue
            for b in range(nb):
                buf, ph = done % bufs, done // bufs
                yield ("wait", f"sf{t}{buf}", ph)
                if not alias:
                    yield ("arrive", f"sr{t}{buf}")
                if masked or b == nb - 1:
                    yield ("wait", f"full{i % ring}", i // ring)
                if done >= bufs:
                    yield ("wait", f"od{t}{buf}", ph - 1)
                if b and (done * 7 + t) % 3 == 0:  # a rescale
                    yield ("wait", f"od{t}{(done - 1) % bufs}", (done - 1) // bufs)
                yield ("arrive", f"pf{t}{buf}")
                i += 1
                done += 1
            if nb:
                yield ("wait", f"od{t}{(done - 1) % bufs}", (done - 1) // bufs)

    roles = {"issuer0": issuer(0), "issuer1": issuer(1), "loader": loader(), "passing": passing()}
    roles.update({f"softmax{t}": softmax(t) for t in range(tiles)})
    return roles, bars


UNITS = [(3, 4, False), (0, 4, False), (1, 2, True), (1, 1, False), (5, 4, True), (2, 3, False), (1, 4, False), (4, 1, True),
         (1, 3, False), (7, 4, False)]


@pytest.mark.parametrize("tiles,ring,bufs,alias", [(4, 4, 1, False), (2, 4, 1, False), (2, 3, 2, True)],
                         ids=["d32", "d64", "d128"])
@pytest.mark.parametrize("seed", range(12))
def test_forward(tiles, ring, bufs, alias, seed):
    units = [(nb, min(rows, tiles), m) for nb, rows, m in UNITS]
    run(*forward(units, tiles, ring, bufs, alias), seed)


def backward(blocks, ring, bufs, groups, dq, units_barrier=True):
    """blocks: of each unit.  dq: the row threads read a row tile, exchange sums and so hold its buffer."""
    bars = {n: Bar(n) for n in ("unit_done",)}
    bars["rest"], bars["epi"] = Bar("rest", groups), Bar("epi", groups)
    for s in range(ring):
        for n in ("land", "full", "empty"):
            bars[f"{n}{s}"] = Bar(f"{n}{s}")
    for x in range(2):
        bars[f"rl{x}"], bars[f"rf{x}"] = Bar(f"rl{x}"), Bar(f"rf{x}")
        bars[f"re{x}"] = Bar(f"re{x}", 1 + groups if dq else 1)
    for x in range(bufs):
        for n in ("sf", "pf", "ad"):
            bars[f"{n}{x}"] = Bar(f"{n}{x}")

    def s_issuer():
        i = use = 0
        for nb in blocks:
            if not nb:
                continue
            yield ("wait", f"rf{use & 1}", use >> 1)
            for b in range(nb):
                yield ("wait", f"full{i % ring}", i // ring)
                if i >= bufs:
                    yield ("wait", f"ad{i % bufs}", i // bufs - 1)
                yield ("arrive", f"sf{i % bufs}")
                if b == nb - 1:
                    yield ("arrive", f"re{use & 1}")
                i += 1
            use += 1

    def sums():
        i = use = 0
        for nb in blocks:
            if nb:
                if use:
                    yield ("wait", "epi", use - 1)
                use += 1
            for b in range(nb):
                yield ("wait", f"pf{i % bufs}", i // bufs)
                yield ("arrive", f"ad{i % bufs}")
                yield ("arrive", f"empty{i % ring}")
                if b == nb - 1:
                    yield ("arrive", "unit_done")
                i += 1

    def loader():
        i = use = 0
        for nb in blocks:
            if not nb:
                continue
            if use >= 2:
                yield ("wait", f"re{use & 1}", (use >> 1) - 1)
            yield ("arrive", f"rl{use & 1}")
            for _ in range(nb):
                if i >= ring:
                    yield ("wait", f"empty{i % ring}", i // ring - 1)
                yield ("arrive", f"land{i % ring}")
                i += 1
            use += 1

    def passing():
        i = use = 0
        for nb in blocks:
            if not nb:
                continue
            yield ("wait", f"rl{use & 1}", use >> 1)
            yield ("arrive", f"rf{use & 1}")
            for _ in range(nb):
                yield ("wait", f"land{i % ring}", i // ring)
                yield ("arrive", f"full{i % ring}")
                i += 1
            use += 1

    def rows(g):
        i = use = 0
        for nb in blocks:
            if not nb:
                continue
            if dq:
                yield ("wait", f"rf{use & 1}", use >> 1)
                yield ("arrive", f"re{use & 1}")
            for _ in range(nb):
                if i % groups == g:
                    yield ("wait", f"sf{i % bufs}", i // bufs)
                    yield ("wait", f"full{i % ring}", i // ring)
                    yield ("arrive", f"pf{i % bufs}")
                i += 1
            if units_barrier:
                yield ("wait", "unit_done", use)
            else:
                yield ("wait", f"ad{(i - 1) % bufs}", (i - 1) // bufs)
            if dq:
                yield ("arrive", "rest")
                yield ("wait", "rest", use)
            yield ("arrive", "epi")
            use += 1

    roles = {"S": s_issuer(), "sums": sums(), "loader": loader(), "passing": passing()}
    roles.update({f"rows{g}": rows(g) for g in range(groups)})
    return roles, bars


BLOCKS = [4, 1, 0, 1, 1, 7, 2, 3, 1, 5, 0, 2]
FORMS = {"d32": (4, 1, 1), "d64": (4, 3, 1), "d128": (3, 2, 2)}  # ring, buffers, groups


@pytest.mark.parametrize("dq", [True, False], ids=["dq", "dkv"])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("seed", range(12))
def test_backward(form, dq, seed):
    run(*backward(BLOCKS, *FORMS[form], dq), seed)


def test_the_last_buffers_barrier_is_not_enough():
    with pytest.raises(ProtocolError, match="EARLY"):
        for seed in range(200):
            run(*backward(BLOCKS, *FORMS["d128"], False, units_barrier=False), seed)

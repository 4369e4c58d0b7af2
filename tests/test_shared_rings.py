"""The rings and barriers of the shared-prefix attention's roles, as a model run under many schedules on
the CPU (tests/test_cache_rings.py has the machine): every wait by parity has to be for the phase that
was meant, no role may wait for ever, and a product reads the tile that it is for."""
import random

import pytest

from tests.test_cache_rings import Bar, Machine, constant, has

FILE = "k_attend_shared.cu"
TWO_BLOCKS, TWO_SLICES, TWO_TILES = range(3)


def model(items, NS, ST, seed, early_free=False, widen=2, quads=2):
    """items: (mode, tiles of stream 0, of stream 1) each.  ``widen`` and ``quads`` warps stand for the
    widening warps and a stream's softmax warps; early_free: a tile is given back with the first stream's
    product, a mistake."""
    JOBS = constant("JOBS", FILE)
    m = Machine(seed)
    full, k_free = [Bar(2) for _ in range(ST)], [Bar(widen) for _ in range(ST)]
    v_full, v_free = [Bar(widen) for _ in range(NS)], [Bar(1) for _ in range(NS)]
    s_full, p_full, o_full, q_full, o_out = ([Bar(c) for _ in range(2)] for c in (2, quads, 1, quads, quads))
    j_full, j_free = [Bar(1) for _ in range(JOBS)], [Bar(2 * quads + widen + 2) for _ in range(JOBS)]
    merge = Bar(2 * quads)
    narrow, wide, out = [None] * ST, [None] * NS, [0, 0]

    def count(mode, n):
        return n[0] if mode == TWO_BLOCKS else n[0] + n[1]

    def ring(mode, u, j):
        return j if mode == TWO_BLOCKS else 2 * j + u

    def jobs(role):
        """The items as a role takes them, and gives them back."""
        for i, (mode, *n) in enumerate(items):
            yield "wait", j_full[i % JOBS], i // JOBS
            yield from role(i, mode, n)
            j_free[i % JOBS].arrive()
            yield 0

    def rows():
        for i in range(len(items)):
            if i >= JOBS:
                yield "wait", j_free[i % JOBS], i // JOBS - 1
            j_full[i % JOBS].arrive()
            yield 0

    def loader():
        at = [0]

        def role(i, mode, n):
            for _ in range(count(mode, n)):
                it = at[0]
                st = it % ST
                if it >= ST:
                    yield "wait", k_free[st], it // ST - 1

                def land(st=st, it=it):
                    narrow[st] = it
                    full[st].arrive(landed=[it])
                yield land
                full[st].arrive()
                yield 0
                at[0] += 1
        yield from jobs(role)

    def widener(w):
        at = [0]

        def role(i, mode, n):
            for _ in range(count(mode, n)):
                it = at[0]
                st, s = it % ST, it % NS
                yield "wait", full[st], it // ST
                assert narrow[st] == it and it in m.known
                k_free[st].arrive()
                yield 0
                if it >= NS:
                    yield "wait", v_free[s], it // NS - 1
                wide[s] = it
                v_full[s].arrive(landed=[-1 - it])
                yield 0
                at[0] += 1
        yield from jobs(role)

    def mma():
        at, pc = [0], [0, 0]

        def scores(mode, u, j, seen=False):
            i = at[0] + ring(mode, u, j)
            if not seen:
                yield "wait", v_full[i % NS], i // NS
            assert wide[i % NS] == i, "scores of another tile"
            yield lambda: s_full[u].arrive()
            s_full[u].arrive()
            yield 0

        def role(item, mode, n):
            for u in range(2):
                if mode == TWO_BLOCKS and u == 0 and n[0]:
                    i = at[0]
                    yield "wait", v_full[i % NS], i // NS
                yield "wait", q_full[u], item
                if n[u]:
                    yield from scores(mode, u, 0, mode == TWO_BLOCKS)
                else:
                    o_full[u].arrive()
                    yield 0
            for j in range(n[0]):
                for u in range(2):
                    if j >= n[u]:
                        break
                    i = at[0] + ring(mode, u, j)
                    if mode == TWO_BLOCKS and u == 0 and j + 1 < n[u]:  # (for both streams)
                        yield "wait", v_full[(i + 1) % NS], (i + 1) // NS
                    yield "wait", p_full[u], pc[u]
                    pc[u] += 1
                    assert wide[i % NS] == i, "a product of another tile"

                    def done(i=i, u=u, free=mode != TWO_BLOCKS or u == 1 or early_free, last=j + 1 == n[u]):
                        assert wide[i % NS] == i, "a tile that is written while it is read"
                        if free and (not early_free or mode != TWO_BLOCKS or u == 0):
                            v_free[i % NS].arrive()
                        if last:
                            o_full[u].arrive()
                    yield done
                    yield 0
                    if j + 1 < n[u]:
                        yield from scores(mode, u, j + 1, mode == TWO_BLOCKS)
            at[0] += count(mode, n)
        yield from jobs(role)

    def soft(u):
        at, sc, mc = [0], [0], [0]

        def role(item, mode, n):
            if item:
                yield "wait", o_out[u], item - 1
            assert not out[u], "queries where O is on its way out"
            q_full[u].arrive()
            yield 0
            for j in range(n[u]):
                i = at[0] + ring(mode, u, j)
                yield "wait", s_full[u], sc[0]
                sc[0] += 1
                assert wide[i % NS] == i and -1 - i in m.known, "the scales of another tile"
                p_full[u].arrive()
                yield 0
            yield "wait", o_full[u], item
            out[u] += 1
            yield 0
            out[u] -= 1
            at[0] += count(mode, n)
            if mode == TWO_TILES:
                for _ in range(2):
                    merge.arrive()
                    yield "wait", merge, mc[0]
                    mc[0] += 1
            o_out[u].arrive()
            yield 0
        yield from jobs(role)

    m.add(rows())
    m.add(loader())
    for w in range(widen):
        m.add(widener(w))
    m.add(mma())
    for u in range(2):
        for _ in range(quads):
            m.add(soft(u))
    m.run()


def some_items(rng):
    out = []
    for _ in range(rng.choice([1, 2, 6])):
        mode = rng.choice([TWO_BLOCKS, TWO_SLICES, TWO_TILES])
        n = rng.choice([1, 1, 2, 3, 7, 12])
        out.append((mode, n, n - (mode == TWO_TILES and rng.random() < 0.5)))
    return out


@pytest.mark.parametrize("dh", [128, 64])
def test_every_role_sees_its_phases(dh):
    text = "NS = DH == 128 ? %d : %d, ST = DH == 128 ? %d : %d"
    assert has(FILE, text % (3, 5, 2, 4)), "the rings' sizes"
    NS, ST = (3, 2) if dh == 128 else (5, 4)
    for seed in range(250):
        model(some_items(random.Random(seed)), NS, ST, seed)


def test_the_model_finds_a_tile_that_is_given_back_too_early():
    with pytest.raises(AssertionError):
        for seed in range(250):
            model(some_items(random.Random(seed)), 3, 2, seed, early_free=True)

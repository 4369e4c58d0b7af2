"""The rings and barriers of the attention kernels' roles, as a model run under many schedules on the
CPU.

A wait for a barrier's phase is by parity: it passes as soon as the barrier's current phase has the
other one, so it means the phase that was meant only where the waiter knows that the phase before has
completed.  The model's roles wait and arrive as the kernels' do (ring sizes and warp counts are read
from the sources); the scheduler holds back some roles, copies and products for long, and every wait
that passes is checked against the phase that it was meant for.  What a copy has written is visible to
those that waited for it, or for a thread that had and then arrived; the arrival of a product's commit
says nothing of the copies before it."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_decode_layer_mxfp8_gb300", "csrc")


def constant(name, file, which=0):
    """A constant of a source; which: 0 the only value, or the wide (1) or narrow (2) form's."""
    text = open(os.path.join(CSRC, file)).read()
    got = re.search(rf"\b{name} = (?:WIDE \? (\d+) : (\d+)|(\d+))\b", text)
    return int(got.group(3) or got.group(which))


def has(file, text):
    """Whether a source says so: what the models' roles do where its kernels once did otherwise."""
    return text in open(os.path.join(CSRC, file)).read()


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase, self.carries = count, 0, 0, set()

    def arrive(self, n=1, landed=()):
        self.carries |= Machine.known
        self.carries.update(landed)
        self.pending += n
        assert self.pending <= self.count, "more arrivals than a phase has"
        if self.pending == self.count:
            self.pending, self.phase = 0, self.phase + 1


class Machine:
    known = set()  # tiles whose copies the running role knows to have landed

    """Roles are generators of ("wait", bar, k): for phase k, by parity; ("sync", bar, k): exactly;
    ("tell", bar, k): nothing passes, k has to be complete; and of functions to call later, in the
    issuing role's order."""

    def __init__(self, seed):
        self.rng, self.roles = random.Random(seed), []

    def add(self, role):
        self.roles.append(role)

    def run(self):
        rng = self.rng
        lazy = rng.choice([0.02, 0.3, 1.0])
        weight = {r: rng.choice([0.02, 0.3, 1.0]) for r in self.roles}
        at, queue = dict.fromkeys(self.roles), {r: [] for r in self.roles}
        known = {r: set() for r in self.roles}
        while at or any(queue.values()):
            can = [(weight[r], r, None) for r, op in at.items() if op is None or self.passes(*op)]
            can += [(lazy, None, q) for q in queue.values() if q]
            assert can, "every role waits"
            _, r, q = rng.choices(can, [c[0] for c in can])[0]
            Machine.known = set() if q else known[r]
            if q:
                q.pop(0)()
                continue
            if at[r] is not None:
                kind, bar, k = at[r]
                assert bar.phase > k, "a wait passed ahead of its phase"
                known[r] |= bar.carries
            op = next(r, None)
            while callable(op):
                queue[r].append(op)
                op = next(r, None)
            if op is None:
                del at[r]
            else:
                at[r] = op or None  # (0: nothing to wait for)

    @staticmethod
    def passes(kind, bar, k):
        return kind == "tell" or (bar.phase > k if kind == "sync" else (bar.phase & 1) != (k & 1))


# ------------------------------------------------------------------ the gathering of weights
WEIGHTS = "k_attend_weights.cu"
TOLD = "mbar_arrive(&ss.s_full[b])"  # the issuing thread arrives for scores, beside their commit


def weights_model(items, chunks, lg, by_slot, both, seed):
    """items: (tiles, passes) each; by_slot: a slot of the ring has one loading warp; both: either MMA
    warp waits for every tile and gives it back."""
    ST, LOADERS, MMAS = (constant(n, WEIGHTS) for n in ("ST", "LOAD_WARPS", "S_WARPS"))
    GROUPS = 4
    told = has(WEIGHTS, TOLD)
    m = Machine(seed)
    full, k_free = [Bar(2) for _ in range(ST)], [Bar(1 + (MMAS if both else 1)) for _ in range(ST)]
    s_full, s_free = [Bar(1 + told) for _ in range(2 * GROUPS)], [Bar(1) for _ in range(2 * GROUPS)]
    holds = [None] * ST  # the tile whose codes, scales and bits a slot holds
    q_full, mma_sync, soft_sync = Bar(GROUPS), Bar(MMAS), Bar(GROUPS)

    def walk(n):  # (place in a row, chunk, first tile of the row, its width)
        for i in range(0, n, GROUPS):
            width = min(GROUPS, n - i)
            for c in range(chunks):
                for tile in range(width):
                    yield tile, c, i, width

    def loader(w):
        it = 0
        for n, passes in items:
            for _ in range(passes):
                for _ in walk(n):
                    s = it % ST
                    if (s if by_slot else it) % LOADERS == w:
                        if it >= ST:
                            yield "wait", k_free[s], it // ST - 1

                        def land(s=s, it=it):
                            holds[s] = it
                            full[s].arrive(landed=[it])
                        yield land
                        full[s].arrive()
                        yield 0
                    it += 1

    def mma(w):
        it, done, used = 0, 0, [0] * GROUPS
        for n, passes in items:
            for _ in range(passes):
                yield "wait", q_full, done
                done += 1
                mma_sync.arrive()
                yield "sync", mma_sync, done - 1
                for tile, _, _, _ in walk(n):
                    st = it % ST
                    if both or tile & 1 == w:
                        yield "wait", full[st], it // ST
                    if tile & 1 != w:
                        if both:
                            k_free[st].arrive()
                    else:
                        assert holds[st] == it, "a product of another tile"
                        k = used[tile]
                        used[tile] += 1
                        b = tile + (k & lg) * GROUPS
                        if k >> lg:
                            yield "wait", s_free[b], (k >> lg) - 1
                        if told:
                            s_full[b].arrive()

                        def done_(b=b, st=st):
                            s_full[b].arrive()
                            k_free[st].arrive()
                        yield done_
                        yield 0
                    it += 1

    def soft(g):
        it, k, done = 0, 0, 0
        for n, passes in items:
            for _ in range(passes):
                soft_sync.arrive()
                yield "sync", soft_sync, done
                done += 1
                q_full.arrive()
                for i in range(0, n, GROUPS):
                    width = min(GROUPS, n - i)
                    for c in range(chunks):
                        if g < width:
                            b, at = g + (k & lg) * GROUPS, it + c * width + g
                            yield "wait", s_full[b], k >> lg
                            assert holds[at % ST] == at and at in m.known, "the bits of another tile"
                            k_free[at % ST].arrive()
                            yield 0
                            s_free[b].arrive()
                            k += 1
                    it += chunks * width

    for w in range(LOADERS):
        m.add(loader(w))
    for w in range(MMAS):
        m.add(mma(w))
    for g in range(GROUPS):
        m.add(soft(g))
    m.run()


def run_weights(chunks, lg, by_slot, both):
    for seed in range(60):
        rng = random.Random(seed)
        weights_model([(rng.choice([1, 2, 3, 4, 5, 7, 9]), rng.choice([1, 1, 2, 3])) for _ in range(3)],
                      chunks, lg, by_slot, both, seed)


@pytest.mark.parametrize("lg", [0, 1])
@pytest.mark.parametrize("chunks", [1, 2, 4, 8])
def test_weights_tiles_are_loaded_into_free_slots(chunks, lg):
    run_weights(chunks, lg, has(WEIGHTS, "it % ST % LOAD_WARPS"), True)


@pytest.mark.parametrize("lg", [0, 1])
@pytest.mark.parametrize("chunks", [1, 2, 4, 8])
def test_weights_products_wait_for_their_own_tiles(chunks, lg):
    run_weights(chunks, lg, True, has(WEIGHTS, "mbar_init(&ss.k_free[s], S_WARPS + 4)"))


# ------------------------------------------------------------------------------ the attention
def attend_model(wide, items, seed):
    """items: (tiles, columns) each.  A softmax group's four warps are one role (they meet at every
    tile), the warps that make queries and widen tiles another."""
    F, which = "k_attend.cu", 1 if wide else 2
    ST, MMAS = constant("ST", F, which), constant("MMA_WARPS", F, which)
    LOADERS, GROUPS = constant("LOAD_WARPS", F), 4
    told = has(F, TOLD)
    by_slot = has(F, "s + LOAD_WARPS < ST ? LOAD_WARPS : ST - s + lw")
    m = Machine(seed)
    full = [Bar(2) for _ in range(ST)]
    k_free = [Bar(2 + 4 if wide else 1) for _ in range(ST)]
    s_full, pv_done, p_full = ([Bar(c) for _ in range(8)] for c in (1 + told, 1, 4))
    v_full, v_free = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
    q_full, q_free = [Bar(1), Bar(1)], [Bar(MMAS), Bar(MMAS)]
    m_free = [Bar(MMAS + GROUPS), Bar(MMAS + GROUPS)]
    o_free, s_sync, soft_sync = Bar(GROUPS), Bar(MMAS), Bar(GROUPS)
    holds = [None] * ST

    class Deal:
        def __init__(self, cols):
            self.lg = 2 if cols <= 16 else 1 if cols <= 32 else 0
            self.streams, self.bufs = 1 << self.lg, 2 << self.lg

        def slot(self, i):
            return i & (self.bufs - 1)

    class Phases:  # of the eight slots, and their change over an item of n tiles
        def __init__(self):
            self.p = [0] * 8

        def of(self, d, i):
            return self.p[d.slot(i)] + (i >> (d.lg + 1))

        def advance(self, d, n):
            for b in range(d.bufs):
                self.p[b] += (n + d.bufs - 1 - b) >> (d.lg + 1)

    total = sum(n for n, _ in items)

    def loader(w):
        for it in range(total):
            s = it % ST
            if (s if by_slot else it) % LOADERS != w:
                continue
            if it >= ST:
                yield "wait", k_free[s], it // ST - 1

            def land(s=s, it=it):
                holds[s] = it
                full[s].arrive(landed=[it])
            yield land
            full[s].arrive()
            yield 0

    def prep():
        it, before = 0, False
        for item, (n, cols) in enumerate(items):
            qb = item & 1
            if item >= 2:
                yield "wait", q_free[qb], (item >> 1) - 1
                yield "wait", m_free[qb], (item >> 1) - 1
            if item > 0 and (cols > 32 or before):
                yield "wait", q_free[qb ^ 1], (item - 1) >> 1
            before = cols > 32
            q_full[qb].arrive()
            if not wide:
                continue
            for _ in range(n):
                s, b = it % ST, it & 1
                yield "wait", full[s], it // ST
                if it >= 2:
                    yield "wait", v_free[b], (it >> 1) - 1
                assert holds[s] == it
                v_full[b].arrive()
                k_free[s].arrive()
                yield 0
                it += 1

    def first(w):
        it, ph = 0, Phases()
        for item, (n, cols) in enumerate(items):
            qb, d = item & 1, Deal(cols)
            yield "wait", q_full[qb], item >> 1
            for i in range(w, n, MMAS):
                st, b = (it + i) % ST, d.slot(i)
                yield "wait", full[st], (it + i) // ST
                assert holds[st] == it + i, "a product of another tile"
                if i >= d.bufs:
                    yield "wait", pv_done[b], ph.of(d, i - d.bufs)
                if told:
                    s_full[b].arrive()

                def done(b=b, st=st):
                    s_full[b].arrive()
                    if wide:
                        k_free[st].arrive()
                yield done
                yield 0
            yield lambda qb=qb: q_free[qb].arrive()
            mine = [i for i in range(max(0, n - MMAS), n) if i % MMAS == w]
            for i in mine:
                yield "wait", pv_done[d.slot(i)], ph.of(d, i)
            s_sync.arrive()  # (behind it, the other warps' last tiles are known to be done)
            yield "sync", s_sync, item
            it += n
            ph.advance(d, n)

    def second(w):
        it, ph = 0, Phases()
        for item, (n, cols) in enumerate(items):
            d = Deal(cols)
            yield "wait", q_full[item & 1], item >> 1
            m_free[item & 1].arrive()
            step = 1 if d.streams == 1 else MMAS
            start = w if w < step else n
            if item > 0 and start < n:
                yield "wait", o_free, item - 1
            for i in range(start, n, step):
                b, st = d.slot(i), (it + i) % ST
                yield "wait", p_full[b], ph.of(d, i)
                if wide:
                    yield "wait", v_full[(it + i) & 1], (it + i) >> 1

                def done(b=b, st=st, v=(it + i) & 1):
                    pv_done[b].arrive()
                    (v_free[v] if wide else k_free[st]).arrive()
                yield done
                yield 0
            it += n
            ph.advance(d, n)

    def soft(g):
        it, ph = 0, Phases()
        for item, (n, cols) in enumerate(items):
            d = Deal(cols)
            yield "wait", q_full[item & 1], item >> 1
            share = 24 if wide and cols > 64 else 16
            stream, c0 = g & (d.streams - 1), (g >> d.lg) * share
            last = None
            if c0 < cols:
                for i in range(stream, n, d.streams):
                    b, st = d.slot(i), (it + i) % ST
                    yield "wait", s_full[b], ph.of(d, i)
                    assert holds[st] == it + i and it + i in m.known, "the bits of another tile"
                    arrive = d.streams + (1 if cols == 48 and g == 0 else 0)
                    if wide:
                        k_free[st].arrive(arrive)
                    if i >= d.streams and m.rng.random() < 0.2:  # the reference moves
                        yield "wait", pv_done[d.slot(i - d.streams)], ph.of(d, i - d.streams)
                    yield 0
                    p_full[b].arrive(arrive)
                    last = i
            # the group's own last tile; those of the other groups are theirs to wait for
            if last is not None and last >= n - MMAS:
                yield "wait", pv_done[d.slot(last)], ph.of(d, last)
            soft_sync.arrive()
            yield "sync", soft_sync, item
            for i in range(n):
                yield "tell", pv_done[d.slot(i)], ph.of(d, i)
            it += n
            ph.advance(d, n)
            o_free.arrive()
            m_free[item & 1].arrive()
            yield 0

    for w in range(LOADERS):
        m.add(loader(w))
    m.add(prep())
    for w in range(MMAS):
        m.add(first(w))
        m.add(second(w))
    for g in range(GROUPS):
        m.add(soft(g))
    m.run()


@pytest.mark.parametrize("wide", [False, True], ids=["narrow", "wide"])
def test_attention_rings(wide):
    columns = [16, 32, 48, 64] + ([96] if wide else [])
    for seed in range(400):
        rng = random.Random(seed)
        attend_model(wide, [(rng.choice([1, 2, 3, 4, 5, 8, 13, 20]), rng.choice(columns))
                            for _ in range(4)], seed)

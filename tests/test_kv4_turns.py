"""Roles and barriers of the row-tile cache attention kernel (csrc/kv4_tile.cu), modelled on the CPU.

A CTA works through segments, one after the other.  In each, the expanding
warps fill a ring of stages with K and V tiles, an issuer a Q tile sends the
products S = Q K^T and O += P V, and four softmax warps a Q tile turn S into P.
The model runs these roles as coroutines with random latencies and checks that
every CTA comes to its end, and that nothing is overwritten while it is still
needed.  Barriers are waited for by the parity of a phase, as in the hardware:
such a wait is right only while the other side is less than two phases away.

A segment is (n, na0, na1, split): key tiles, those that Q tile 0 / 1 has rows
for (a prefix), and whether the unit spans CTAs (its end is then a barrier of
all softmax warps).
"""

import heapq
import random

import pytest

GROUP_WARPS = 4                                   # softmax warps of a Q tile


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0   # phase: the one that is under way

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):                     # has the phase of this parity ended?
        return (self.phase & 1) != parity


class Cta:
    def __init__(self, segments, stages, rng, turns="count", together=True, q_tiles=2, slow=None):
        self.segments, self.S, self.rng, self.turns, self.Q = segments, stages, rng, turns, q_tiles
        self.together = together                  # a Q tile without keys takes part in the segment's barriers all the same
        self.slow = slow or {}                    # role -> factor of its delays
        self.now, self.events, self.order, self.blocked = 0.0, [], 0, []
        warps = 4 if q_tiles == 2 else 8
        self.expanders = warps
        self.b_q = [Barrier(GROUP_WARPS) for _ in range(q_tiles)]
        self.b_s = [Barrier(1) for _ in range(q_tiles)]
        self.b_p = [Barrier(GROUP_WARPS) for _ in range(q_tiles)]
        self.full = [Barrier(warps) for _ in range(stages)]
        self.empty = [Barrier(q_tiles) for _ in range(stages)]
        self.soft_sync, self.expand_sync = Barrier(GROUP_WARPS * q_tiles), Barrier(warps)
        self.written = [0] * q_tiles              # warps' P tiles since the beginning
        self.stage = [None] * stages              # (segment, kind, key tile) in each stage
        self.busy = [0] * stages                  # products under way that read it
        self.s = [None] * q_tiles                 # whose scores S holds
        self.o = [None] * q_tiles
        self.q = [None] * q_tiles
        self.dead, self.nan = [None] * 8, [None] * 8
        self.pipe = [0.0] * q_tiles               # when an issuer's last product ends
        self.finished = 0
        roles = [("issuer%d" % q, self.issuer(q)) for q in range(q_tiles)]
        roles += [("soft%d" % q, self.softmax(q)) for q in range(q_tiles) for _ in range(GROUP_WARPS)]
        roles += [("expand", self.expand(w)) for w in range(warps)]
        self.roles = len(roles)
        for name, gen in roles:
            self.step(name, gen)

    # ---- scheduling
    def at(self, t, fn):
        self.order += 1
        heapq.heappush(self.events, (t, self.order, fn))

    def step(self, name, gen):
        try:
            want = next(gen)
        except StopIteration:
            self.finished += 1
            return
        if callable(want):
            self.blocked.append((want, name, gen))
        else:
            d = want * self.rng.uniform(0.7, 1.5) * self.slow.get(name, 1.0)
            self.at(self.now + d, lambda: self.step(name, gen))

    def run(self):
        """True if every role comes to its end."""
        while True:
            ready = [b for b in self.blocked if b[0]()]
            if ready:
                self.blocked = [b for b in self.blocked if b not in ready]
                self.rng.shuffle(ready)
                for _, name, gen in ready:
                    self.step(name, gen)
            elif self.events:
                self.now, _, fn = heapq.heappop(self.events)
                fn()
            else:
                return self.finished == self.roles

    # ---- roles
    def product(self, q, cost, stage, begin, end):
        """A product of issuer q: it reads `stage`, and its issuer's products end in order."""
        begin()
        self.busy[stage] += 1
        self.pipe[q] = max(self.pipe[q], self.now) + cost * self.rng.uniform(0.7, 1.5)

        def done():
            self.busy[stage] -= 1
            end()
        self.at(self.pipe[q], done)

    def commit(self, q, bar):
        self.at(max(self.pipe[q], self.now), bar.arrive)

    def issuer(self, q):
        st, kph, pph, qph = 0, 0, 0, 0

        def advance():
            nonlocal st, kph
            st += 1
            if st == self.S:
                st, kph = 0, kph ^ 1

        def scores(i, j, stage):
            def begin():
                assert self.stage[stage] == (i, "k", j) and self.q[q] == i
                self.s[q] = None
            self.product(q, 300, stage, begin, lambda: self.s.__setitem__(q, (i, j)))
            self.commit(q, self.b_s[q])

        for i, seg in enumerate(self.segments):
            n, na = seg[0], seg[1 + q]
            if n == 0:
                continue
            if na > 0 or self.together:
                ph = qph
                yield lambda: self.b_q[q].passed(ph)
                qph ^= 1
            yield lambda s=st, ph=kph: self.full[s].passed(ph)
            if na > 0:
                scores(i, 0, st)
            elif self.together:
                self.commit(q, self.b_s[q])
            self.commit(q, self.empty[st])
            advance()
            for j in range(n):
                vst = st
                yield lambda s=vst, ph=kph: self.full[s].passed(ph)
                advance()
                if j < na:
                    yield lambda ph=pph: self.b_p[q].passed(ph)
                    pph ^= 1

                    def begin(i=i, j=j, vst=vst):
                        assert self.stage[vst] == (i, "v", j)
                        self.o[q] = None
                    self.product(q, 300, vst, begin, lambda i=i, j=j: self.o.__setitem__(q, (i, j)))
                    if j + 1 == na:
                        self.commit(q, self.b_s[q])
                self.commit(q, self.empty[vst])
                if j + 1 < n:
                    yield lambda s=st, ph=kph: self.full[s].passed(ph)
                    if j + 1 < na:
                        scores(i, j + 1, st)
                    self.commit(q, self.empty[st])
                    advance()

    def softmax(self, q):
        sph, tiles, turns, seen = 0, 0, 0, 0
        for i, seg in enumerate(self.segments):
            n, na = seg[0], seg[1 + q]
            other = seg[2 - q] if self.Q == 2 else 0
            if na > 0:
                yield 1500                        # query rows from memory
                self.q[q] = i
            if na > 0 or (n > 0 and self.together):
                self.b_q[q].arrive()
            for j in range(na):
                yield lambda ph=sph: self.b_s[q].passed(ph)
                sph ^= 1
                assert self.s[q] == (i, j), "scores overwritten"
                k = j - (1 if q == 0 else 0)
                if 0 <= k < other:
                    if self.turns == "parity":
                        yield lambda ph=(turns + k) & 1: self.b_p[1 - q].passed(ph)
                    elif self.turns == "count" or self.rng.random() < 0.5:   # "tries": a wait may be given up
                        yield lambda c=GROUP_WARPS * (turns + k + 1): self.written[1 - q] >= c
                assert self.dead[(tiles + j) % 8] == tiles + j, "notes of a key tile overwritten"
                yield 900
                self.written[q] += 1
                self.b_p[q].arrive()
            if na > 0 or (n > 0 and self.together):
                yield lambda ph=sph: self.b_s[q].passed(ph)
                sph ^= 1
            if na > 0:
                yield 700
                assert self.o[q] == (i, na - 1), "output overwritten"
                assert self.nan[seen % 8] == seen, "notes of a segment overwritten"
            if seg[3]:
                ph = self.soft_sync.phase
                self.soft_sync.arrive()
                yield lambda ph=ph: self.soft_sync.phase > ph
                yield 1000
            tiles += n
            seen += n > 0
            turns += other

    def expand(self, w):
        issued, tiles, seen = 0, 0, 0
        for i, seg in enumerate(self.segments):
            n = seg[0]
            if n == 0:
                continue
            self.nan[seen % 8] = seen
            ph = self.expand_sync.phase
            self.expand_sync.arrive()
            yield lambda ph=ph: self.expand_sync.phase > ph
            yield 600                             # page numbers, first words
            for j in range(n):
                for kind in "kv":
                    st, parity = issued % self.S, ((issued // self.S) & 1) ^ 1
                    yield lambda st=st, parity=parity: self.empty[st].passed(parity)
                    issued += 1
                    assert self.busy[st] == 0, "stage overwritten"
                    self.stage[st] = (i, kind, j)
                    if kind == "k":
                        self.dead[(tiles + j) % 8] = tiles + j
                    yield 250
                    self.full[st].arrive()
            tiles += n
            seen += 1


def runs(segments, stages, seed, **kw):
    return Cta(segments, stages, random.Random(seed), **kw).run()


# ------------------------------------------------------------------ what a call gives each CTA

def parts(lens, qlens, Hq, Hkv, ctas=152, q_tiles=2, causal=True, split_rows=96):
    """Segments of each CTA: the line of work of csrc/kv4_walk.cuh, written out."""
    G, rows_of, keys = Hq // Hkv, 128 * q_tiles, 128
    line = []                                     # (places of the unit, blocks, limit, limits of its Q tiles)
    for L, n in zip(lens, qlens):
        rows = n * G
        if rows < split_rows:
            continue
        blocks = max(1, -(-L // keys))
        see = lambda row: max(0, min(L, L - n + row // G + 1)) if causal else L
        for rt in range(-(-rows // rows_of)):
            here = min(rows_of, rows - rt * rows_of)
            lims = [see(rt * rows_of + min(here, 128 * (q + 1)) - 1) if here > 128 * q else 0 for q in range(2)]
            line += [(blocks + 1, blocks, see(rt * rows_of + here - 1), lims)] * Hkv
    total = sum(u[0] for u in line)
    cut = min(ctas, total)
    ends = [(total // cut) * (c + 1) + min(c + 1, total % cut) for c in range(cut)]
    out, pos, c = [[] for _ in range(cut)], 0, 0
    for size, blocks, limit, lims in line:
        first, blk = pos + 1, 0
        while blk < blocks:
            while ends[c] <= first + blk:
                c += 1
            nb = min(blocks - blk, ends[c] - first - blk)
            tiles = lambda lim: max(0, min(nb, -(-(lim - blk * keys) // keys)))
            out[c].append((tiles(limit), tiles(lims[0]), tiles(lims[1]), nb < blocks))
            blk += nb
        pos += size
    return out


MIXES = [
    [(2, 1, 2, False)] * 12,                      # 256-token prompts without grouped heads
    [(3, 3, 0, False)] * 3 + [(3, 3, 3, False)] * 3,
    [(4, 4, 0, False)] * 9 + [(2, 2, 2, False)] * 4,
    [(1, 1, 0, False)] * 20 + [(5, 4, 5, True)] * 3,
    [(4, 3, 4, False), (1, 1, 0, False)] * 6,
    [(1, 0, 1, False), (2, 2, 2, False)] * 6,     # rows without keys in the first Q tile
    [(0, 0, 0, False), (2, 1, 2, True), (0, 0, 0, True)] * 5,
    [(7, 6, 7, False), (6, 6, 6, True), (3, 3, 0, False)] * 4,
    [(9, 2, 9, False), (9, 9, 9, False)] * 3,
]
CALLS = {
    "32 prompts of 256 tokens": ([256] * 32, [256] * 32, 32, 32),
    "16 prompts of 1000 tokens": ([1000] * 16, [1000] * 16, 32, 32),
    "16 parts of 280 tokens over 900": ([900] * 16, [280] * 16, 32, 8),
    "64 parts of 90 tokens over 600": ([600] * 64, [90] * 64, 32, 8),
    "48 prompts of mixed lengths": ([50 + 41 * i for i in range(48)], [50 + 41 * i for i in range(48)], 32, 8),
}


@pytest.mark.parametrize("turns", ["count", "tries"])
@pytest.mark.parametrize("stages", [5, 8])
@pytest.mark.parametrize("mix", range(len(MIXES)))
def test_every_mix_of_segments_comes_to_its_end(mix, stages, turns):
    for seed in range(30):
        assert runs(MIXES[mix], stages, seed, turns=turns)


@pytest.mark.parametrize("role", ["soft0", "soft1", "issuer0", "issuer1", "expand"])
def test_slow_roles(role):
    for mix in MIXES:
        for seed in range(4):
            for stages in (5, 8):
                assert runs(mix, stages, seed, turns=("count", "tries")[seed % 2], slow={role: 20.0})


@pytest.mark.parametrize("stages", [5, 8])
def test_random_mixes(stages):
    rng = random.Random(stages)
    for seed in range(150):
        segs = []
        for _ in range(rng.randrange(1, 14)):
            n = rng.choice([0, 1, 1, 2, 3, 4, 6])
            segs.append((n, rng.randint(0, n), rng.randint(0, n), rng.random() < 0.2))
        segs = [(max(a, b), a, b, s) for _, a, b, s in segs]
        assert runs(segs, stages, seed, turns=("count", "tries")[seed % 2]), segs


@pytest.mark.parametrize("name", list(CALLS))
def test_calls_of_many_requests(name):
    """Every CTA of a call; at head_dim 128 (5 stages) and 64 (8 stages)."""
    for c, segs in enumerate(parts(*CALLS[name])):
        assert len(segs) > 0
        assert runs(segs, 5 if c % 2 else 8, c, turns=("tries", "count")[c % 3 == 0])


def test_parity_alone_would_stall():
    """Why the turns are counted: a Q tile that is two phases ahead looks like one that has not come."""
    assert sum(not runs(MIXES[0], 5, seed, turns="parity") for seed in range(30)) > 20
    assert sum(not runs(MIXES[1], 5, seed, turns="parity") for seed in range(30)) > 20
    # within one segment, and where every segment ends in a barrier, parity is enough
    assert all(runs([(40, 39, 40, True)], 5, seed, turns="parity") for seed in range(5))
    assert all(runs([(3, 3, 3, True)] * 8, 5, seed, turns="parity") for seed in range(10))


def test_a_q_tile_without_keys_stays_with_the_others():
    """Else the other one passes segments by the dozen while its last output is still being written."""
    segs = [(1, 1, 1, False)] + [(1, 1, 0, False)] * 20
    for seed in range(10):
        assert runs(segs, 8, seed, slow={"soft1": 60.0})
        with pytest.raises(AssertionError, match="notes of a segment"):
            runs(segs, 8, seed, slow={"soft1": 60.0}, together=False)


def test_one_q_tile():
    for seed in range(20):
        segs = [(3, 3, 0, False), (1, 1, 0, True), (0, 0, 0, False), (5, 5, 0, False)] * 3
        assert runs(segs, 2, seed, q_tiles=1)

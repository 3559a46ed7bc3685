"""Host model of a tree attention CTA from segment to segment (csrc/tree.cu), in the kernel's own order.

test_tree_protocol.py covers the ring of tiles inside a run. Here are the roles as they go on from one
segment to the next: the planner and its ring of segments, which seven readers release; the copies, which
note tiles with a bad page; two issuers, whose products complete some time after they are issued; and
four softmax warps, which at a segment's end write the next one's queries, wait for the last product,
arrive for the next scores, and only then read the outputs, while those scores may run. Infinite or NaN
elements of new values are reported through one word of shared memory.

Each role is a generator that gives way before every access to what others share. Schedules are random,
some roles being slow in some of them.
"""
import random

import pytest

from test_pipeline_protocol import Barrier

NB, NG, W = 3, 4, 4


class Cta:
    def __init__(self, segments, seed, NS=5, notes=16, fault=None):
        """segments: a list a segment of (tail, odd, bad) a tile: V is mended; it holds elements that are not
        finite; its page is bad."""
        self.rng = random.Random(seed)
        self.segments, self.NS, self.notes, self.fault = segments, NS, notes, fault
        self.tiles = [(s, i) + t for s, seg in enumerate(segments) for i, t in enumerate(seg)]
        self.T = len(self.tiles)
        self.full, self.empty = ([Barrier(1) for _ in range(NS)] for _ in range(2))
        self.q_full, self.v_ready = Barrier(W), Barrier(W)
        self.s_full, self.pv_done = ([Barrier(1) for _ in range(NB)] for _ in range(2))
        self.p_full = [Barrier(W) for _ in range(NB)]
        self.g_full = [Barrier(1) for _ in range(NG)]
        self.g_empty = [Barrier(6 if fault == "a reader too few" else 7) for _ in range(NG)]
        self.ring, self.slot, self.cols, self.note = [None] * NG, [None] * NS, [None] * NB, [0] * notes
        self.queries, self.outputs, self.flag = [None] * W, None, 0
        self.landing, self.products = [], [[], []]
        self.weights, self.read, self.fixed = [0] * self.T, [0] * len(segments), [0] * self.T
        self.scores_left = [len(s) for s in segments]
        self.running = 0

    def k_at(self, i):
        return 0 if i == 0 else 2 * i - 1

    def v_at(self, i):
        return 2 * i + 2 if i + 1 < self.T else 2 * i + 1

    def wait(self, bar, n):
        while not bar.test(n):
            yield False
        yield True

    def segment(self, i):
        yield from self.wait(self.g_full[i % NG], i // NG)
        g = self.ring[i % NG]
        assert g == (i if i < len(self.segments) else "end"), "a segment that was overwritten"
        return g

    # ------------------------------------------------------------------ roles
    def planner(self):
        for i in range(len(self.segments) + 1):
            if i >= NG:
                yield from self.wait(self.g_empty[i % NG], i // NG - 1)
            self.ring[i % NG] = i if i < len(self.segments) else "end"
            yield True
            self.g_full[i % NG].arrive(i // NG)

    def look_up(self, i):
        """The copies' view of tile i, looked up a tile ahead."""
        s, first = self.tiles[i][0], self.tiles[i][1] == 0
        if first:
            yield from self.segment(s)
            self.g_empty[s % NG].arrive(s // NG)

    def copies(self):
        yield from self.look_up(0)
        for at in range(2 * self.T):
            i = (at + 1) // 2
            if at == 0 or (at & 1 and i < self.T):
                load = ("K", i)
                if self.tiles[i][4]:
                    self.note[i % self.notes] = i + 1
                yield True
                if i + 1 < self.T:
                    yield from self.look_up(i + 1)
            else:
                load = ("V", i - 1)
            if at >= self.NS:
                yield from self.wait(self.empty[at % self.NS], at // self.NS - 1)
            self.slot[at % self.NS] = None
            self.landing.append((at, load))
            yield True

    def land(self):
        while True:
            if self.landing:
                at, load = self.landing.pop(self.rng.randrange(len(self.landing)))
                self.slot[at % self.NS] = load
                self.full[at % self.NS].arrive(at // self.NS)
            yield bool(self.landing)

    def issue_scores(self):
        for i, (s, k, *_) in enumerate(self.tiles):
            if k == 0:
                yield from self.segment(s)
                self.g_empty[s % NG].arrive(s // NG)
                if self.fault != "scores without queries":
                    yield from self.wait(self.q_full, s)
            if i >= NB:
                yield from self.wait(self.pv_done[i % NB], i // NB - 1)
            yield from self.wait(self.full[self.k_at(i) % self.NS], self.k_at(i) // self.NS)
            self.products[0].append(i)
            yield True

    def issue_outputs(self):
        for i, (s, k, *_) in enumerate(self.tiles):
            if k == 0:
                yield from self.segment(s)
                self.g_empty[s % NG].arrive(s // NG)
            yield from self.wait(self.full[self.v_at(i) % self.NS], self.v_at(i) // self.NS)
            yield from self.wait(self.p_full[i % NB], i // NB)
            self.products[1].append(i)
            yield True

    def tensor_cores(self, kind):
        """One issuer's products, which complete in order: operands are read from the issue to the end."""
        while True:
            while not self.products[kind]:
                yield False
            i = self.products[kind][0]
            s, k, tail, odd, _ = self.tiles[i]
            at = self.v_at(i) if kind else self.k_at(i)

            def operands():
                assert self.slot[at % self.NS] == ("KV"[kind], i), "a tile that is not there"
                if kind:
                    assert self.cols[i % NB] == ("P", i) and self.weights[i] == W, "weights that are not there"
                    assert not tail or self.fixed[i] == W, "values that are not mended"
                    assert k or all(n == W for n in self.read[:s]), "outputs overwritten before they are read"
                else:
                    assert self.queries == [s] * W, "scores of other queries"
            operands()
            if kind:
                self.outputs = (s, "partly")
            else:
                self.cols[i % NB] = None
            yield True
            operands()
            if kind:
                self.outputs = (s, k)
            else:
                self.cols[i % NB] = ("S", i)
                self.scores_left[s] -= 1
            self.products[kind].pop(0)
            self.empty[at % self.NS].arrive(at // self.NS)
            (self.pv_done if kind else self.s_full)[i % NB].arrive(i // NB)
            yield True

    def softmax(self, n):
        i, tails, rescales = 0, 0, self.rng.random()

        def read_outputs(s, last):
            for _ in range(3):
                assert self.outputs == (s, last), "outputs of other tiles"
                yield True
            self.read[s] += 1
        yield from self.segment(0)
        self.g_empty[0].arrive(0)
        self.queries[n] = 0
        yield True
        self.q_full.arrive(0)
        late = None
        for s, tiles in enumerate(self.segments):
            bad = False
            for k, (tail, odd, is_bad) in enumerate(tiles):
                yield from self.wait(self.s_full[i % NB], i // NB)
                assert self.cols[i % NB] == ("S", i) or self.weights[i]
                assert (self.note[i % self.notes] == i + 1) == is_bad, "a note that was overwritten"
                bad |= is_bad
                if k and self.rng.random() < rescales:
                    yield from self.wait(self.pv_done[(i - 1) % NB], (i - 1) // NB)
                    assert self.outputs == (s, k - 1)
                if tail:
                    at = self.v_at(i)
                    yield from self.wait(self.full[at % self.NS], at // self.NS)
                    assert self.slot[at % self.NS] == ("V", i)
                    if odd and n == i % W:  # this warp's rows of V hold it
                        self.flag = s + 1
                    self.fixed[i] += 1
                    yield True
                    self.v_ready.arrive(tails)
                    yield from self.wait(self.v_ready, tails)
                    assert self.fixed[i] == W
                    tails += 1
                self.weights[i] += 1
                if self.weights[i] == W:
                    self.cols[i % NB] = ("P", i)
                yield True
                self.p_full[i % NB].arrive(i // NB)
                if late:
                    yield from late
                    late = None
                i += 1
            assert bad == any(t[2] for t in tiles)
            more = (yield from self.segment(s + 1)) != "end"
            if more:
                self.g_empty[(s + 1) % NG].arrive((s + 1) // NG)
                assert self.scores_left[s] == 0, "queries overwritten under products"
                self.queries[n] = s + 1
                yield True
            yield from self.wait(self.pv_done[(i - 1) % NB], (i - 1) // NB)
            odd = self.flag == s + 1
            yield True
            if more:
                self.q_full.arrive(s + 1)
                yield True
            if self.fault == "flag read late":
                odd = self.flag == s + 1
            assert odd == any(t[1] for t in tiles), "the flag of another segment"
            if self.fault == "outputs read late" and more:
                late = read_outputs(s, len(tiles) - 1)
            else:
                yield from read_outputs(s, len(tiles) - 1)
        self.running -= 1

    def run(self):
        warps = [self.softmax(n) for n in range(W)]
        roles = [self.planner(), self.copies(), self.land(), self.issue_scores(), self.issue_outputs(), self.tensor_cores(0),
                 self.tensor_cores(1)] + warps
        pace = [self.rng.choice([1.0, 1.0, 0.3, 0.03]) for _ in roles]
        self.running, idle, over = W, 0, set()
        while self.running:
            r = self.rng.choices(range(len(roles)), pace)[0]
            if r in over:
                continue
            try:
                moved = next(roles[r])
            except StopIteration:
                over.add(r)
                continue
            idle = 0 if moved else idle + 1
            assert idle < 50000, "no role can move"
        assert self.read == [W] * len(self.segments)


def tiles_of(sizes, seed):
    """Runs of segments: tiles at a sequence's end (new tokens) are mended, some hold what is not finite."""
    rng = random.Random(seed)
    out = []
    for n in sizes:
        ends = rng.randint(0, 2)
        out.append([(i >= n - ends, i >= n - ends and rng.random() < 0.5, rng.random() < 0.1) for i in range(n)])
    return out


SHAPES = [[1], [3], [40], [1] * 9, [2, 1, 3, 1, 1, 2], [7, 1, 1, 9], [1, 20, 1, 1, 1, 1, 5]]


@pytest.mark.parametrize("NS", [5, 6, 8])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_roles_agree_from_segment_to_segment(NS, shape):
    for seed in range(15):
        Cta(tiles_of(shape, seed), seed, NS).run()


FAULTS = {"flag read late": "the flag of another segment", "outputs read late": "outputs",
          "a reader too few": "overwritten|phase", "scores without queries": "other queries"}


@pytest.mark.parametrize("fault", FAULTS)
def test_the_model_catches(fault):
    """Each of these in the kernel's place: the flag read after the arrival that lets the next segment's scores run;
    weights announced before the outputs are read; a ring of segments that counts six of its seven readers;
    scores that do not wait for queries."""
    with pytest.raises(AssertionError, match=FAULTS[fault]):
        for seed in range(400):
            Cta([[(True, True, False)]] * 12, seed, fault=fault).run()


def test_the_model_catches_notes_that_are_too_few():
    with pytest.raises(AssertionError, match="a note that was overwritten"):
        for seed in range(200):
            Cta([[(False, False, i % 2 == 0) for i in range(30)]], seed, NS=8, notes=2).run()

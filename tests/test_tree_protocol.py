"""Host model of the tree attention's barriers (csrc/tree.cu), run under random interleavings of
its roles, and of how runs of tiles are cut and their parts found again.

A CTA takes a run of key tiles that goes through several segments (items or parts of them). K and V
tiles pass through one ring of slots in the order K0 K1 V0 K2 V1 ... that ignores where segments
end. One thread issues the scores' products (once a segment's queries are there), another the outputs'
in place of them, and four softmax warps turn a tile's scores into
weights in place, mend V at the end of a sequence, now and then rescale the output, and read it at a
segment's end. An mbarrier tells phases apart by parity alone: Barrier checks that every wait is for the
phase at hand or the one before, and every arrival in its own phase.
"""
import random

import pytest

from test_pipeline_protocol import Barrier

NB = 3


def run(NS, segments, seed, skip=None):
    """segments: tiles of each, with whether a tile is at its sequence's end (V is mended)."""
    rng = random.Random(seed)
    tiles = [(s, i, i == len(t) - 1, tail) for s, t in enumerate(segments) for i, tail in enumerate(t)]
    T = len(tiles)

    def k_at(i):
        return 0 if i == 0 else 2 * i - 1

    def v_at(i):
        return 2 * i + 2 if i + 1 < T else 2 * i + 1
    order = {}
    for i in range(T):
        order[k_at(i)] = ("K", i)
        order[v_at(i)] = ("V", i)
    assert sorted(order) == list(range(2 * T))
    W = 4
    full, empty = [Barrier(1) for _ in range(NS)], [Barrier(1) for _ in range(NS)]
    q_full, v_ready = Barrier(W), Barrier(W)
    s_full, p_full, pv_done = [Barrier(1) for _ in range(NB)], [Barrier(W) for _ in range(NB)], [Barrier(1) for _ in range(NB)]
    slot, cols = [None] * NS, [None] * NB  # what a slot holds; a buffer's scores or weights
    queries, output = [None] * W, None       # the segment whose queries each warp has written, whose outputs there are
    state = dict(load=0, qk=0, pv=0)
    done_pv, mended, coming = -1, set(), []

    def load():
        at = state["load"]
        if at >= 2 * T or (at >= NS and not empty[at % NS].test(at // NS - 1)):
            return False
        slot[at % NS] = None
        coming.append(at)
        state["load"] += 1
        return True

    def land():  # copies end in any order
        if not coming:
            return False
        at = coming.pop(rng.randrange(len(coming)))
        slot[at % NS] = order[at]
        full[at % NS].arrive(at // NS)
        return True

    def qk():
        i = state["qk"]
        if i >= T:
            return False
        seg, first = tiles[i][0], tiles[i][1] == 0
        at = k_at(i)
        if first and skip != "queries" and not q_full.test(seg):
            return False
        if i >= NB and not pv_done[i % NB].test(i // NB - 1) or not full[at % NS].test(at // NS):
            return False
        assert slot[at % NS] == ("K", i) and queries == [seg] * W, "scores of other queries"
        assert i < NB or done_pv >= i - NB, "weights overwritten"
        cols[i % NB] = ("S", i)
        empty[at % NS].arrive(at // NS)
        s_full[i % NB].arrive(i // NB)
        state["qk"] += 1
        return True

    def pv():
        nonlocal done_pv, output
        i = state["pv"]
        if i >= T:
            return False
        seg, k, _, tail = tiles[i]
        at = v_at(i)
        if not full[at % NS].test(at // NS) or not p_full[i % NB].test(i // NB):
            return False
        assert slot[at % NS] == ("V", i) and cols[i % NB] == ("P", i)
        assert not tail or i in mended, "V used before it is mended"
        if k == 0:
            assert all(w["read"] >= seg for w in warps), "outputs overwritten before they are read"
        output = seg
        done_pv = i
        empty[at % NS].arrive(at // NS)
        pv_done[i % NB].arrive(i // NB)
        state["pv"] += 1
        return True

    warps = [dict(i=0, step="queries", read=0, tails=0) for _ in range(W)]
    rescales = [rng.random() < 0.3 for _ in range(T)]
    written, fixed = [0] * T, [0] * T

    def soft(n):
        w = warps[n]
        i = w["i"]
        if i >= T:
            return False
        seg, k, last, tail = tiles[i]
        if w["step"] == "queries":
            if k == 0:
                assert all(tiles[j][0] >= seg for j in range(state["qk"], T)), "queries overwritten under products"
                queries[n] = seg
                q_full.arrive(seg)
            w["step"] = "scores"
        elif w["step"] == "scores":
            if not s_full[i % NB].test(i // NB):
                return False
            if k > 0 and rescales[i]:
                if not pv_done[(i - 1) % NB].test((i - 1) // NB):
                    return False
                assert done_pv == i - 1 and output == seg
            w["step"] = "mend" if tail else "weights"
        elif w["step"] == "mend":
            at = v_at(i)
            if not full[at % NS].test(at // NS):
                return False
            assert slot[at % NS] == ("V", i)
            fixed[i] += 1
            v_ready.arrive(w["tails"])
            w["step"] = "mended"
        elif w["step"] == "mended":
            if not v_ready.test(w["tails"]):
                return False
            assert fixed[i] == W
            mended.add(i)
            w["tails"] += 1
            w["step"] = "weights"
        elif w["step"] == "weights":
            written[i] += 1
            if written[i] == W:
                assert cols[i % NB] == ("S", i)
                cols[i % NB] = ("P", i)
            p_full[i % NB].arrive(i // NB)
            w["step"] = "outputs" if last else "queries"
            if not last:
                w["i"] += 1
        else:
            if not pv_done[i % NB].test(i // NB):
                return False
            assert done_pv == i and output == seg
            w["read"] = seg + 1
            w["i"] += 1
            w["step"] = "queries"
        return True

    roles, idle = [load, land, qk, pv] + [lambda n=n: soft(n) for n in range(W)], 0
    while any(w["i"] < T for w in warps):
        idle = 0 if rng.choice(roles)() else idle + 1
        assert idle < 20000, f"no role can move: {state} {warps}"


SHAPES = [[1], [2], [3], [50], [1, 1], [1, 1, 1, 1, 1], [2, 1, 3], [7, 1, 1, 9], [4, 4, 4], [1, 30, 1]]


@pytest.mark.parametrize("NS", [4, 5, 6, 8])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_barriers_hold_under_random_schedules(NS, shape):
    for seed in range(25):
        rng = random.Random(seed)
        # up to two tiles at a sequence's end hold new tokens
        ends = [rng.randint(0, 2) for _ in shape]
        run(NS, [[i >= n - e for i in range(n)] for n, e in zip(shape, ends)], seed)


def test_the_model_catches_a_ring_that_is_too_short():
    """With three slots V of a tile takes the slot that its own K had: the outputs' issuer may come to wait
    for V's phase before K's is over, and takes the one before for it. (The kernel refuses to compile so.)"""
    with pytest.raises(AssertionError, match="waiting for phase"):
        for seed in range(60):
            run(3, [[False] * 8], seed)
    for seed in range(60):
        run(4, [[False] * 8, [True, True], [False] * 5], seed)


def test_the_model_catches_scores_of_other_queries():
    with pytest.raises(AssertionError):
        for seed in range(60):
            run(6, [[False] * 3] * 6, seed, skip="queries")


# ------------------------------------------------------------------ runs and parts
def begin(total, cta, ctas):
    return min(cta, total) if total <= ctas else total * cta // ctas


class Seq:
    """A sequence's tiles as the kernel numbers them: KV head, chunk of keys, row tile, key."""

    def __init__(self, heads, kt, rt, run):
        self.heads, self.kt, self.rt = heads, kt, rt
        self.chunks = max(1, (2 * kt + run) // (2 * run)) if rt > 1 else 1
        self.count = heads * kt * rt

        self.size, self.longer = divmod(kt, self.chunks) if kt else (0, 0)

    def segment(self, off, left):
        """(head, row tile, k0, k1) of the segment at a tile, at most `left` tiles long."""
        h, at = divmod(off, self.kt * self.rt)
        x, long = at // self.rt, self.longer * (self.size + 1)
        chunk = x // (self.size + 1) if x < long else self.longer + (x - long) // self.size
        lo, n = chunk * self.size + min(chunk, self.longer), self.size + (chunk < self.longer)
        row, k = divmod(at - lo * self.rt, n)
        assert 0 <= row < self.rt and 0 <= chunk < self.chunks
        return h, row, lo + k, min(lo + n, lo + k + left)


def cut(sizes, ctas):
    """Every CTA's segments [(sequence, head, row tile, k0, k1)], and the sequences."""
    total = sum(h * kt * rt for h, kt, rt in sizes)
    run = max(1, -(-total // ctas))
    seqs, out = [Seq(*s, run) for s in sizes], []
    b, base = 0, 0
    for cta in range(ctas):
        at, end, mine = begin(total, cta, ctas), begin(total, cta + 1, ctas), []
        while at < end:
            while at >= base + seqs[b].count:
                base += seqs[b].count
                b += 1
            h, row, k0, k1 = seqs[b].segment(at - base, end - at)
            mine.append((b, h, row, k0, k1))
            at += k1 - k0
        out.append(mine)
    return out, seqs


PARTS = 3


@pytest.mark.parametrize("seed", range(80))
def test_every_tile_once_and_few_parts(seed):
    """Every item's keys are covered once, in order; no CTA has more parts than it has places for."""
    rng = random.Random(seed)
    ctas = rng.choice([1, 2, 7, 152, 160])
    most = rng.choice([1, 3, 20, 300])
    sizes = [(rng.choice([1, 2, 8]), rng.randint(0, 1) and rng.randint(1, most), rng.choice([1, 1, 2, 3, 4, 8]))
             for _ in range(rng.choice([1, 2, 5, 40]))]
    runs, seqs = cut(sizes, ctas)
    got = {}
    for mine in runs:
        assert sum((k0, k1) != (0, seqs[b].kt) for b, _, _, k0, k1 in mine) <= PARTS
        for b, h, row, k0, k1 in mine:
            got.setdefault((b, h, row), []).append((k0, k1))
    for b, (heads, kt, rt) in enumerate(sizes):
        for h in range(heads if kt else 0):
            for row in range(rt):
                parts = got.pop((b, h, row))
                assert parts[0][0] == 0 and parts[-1][1] == kt and all(x[1] == y[0] for x, y in zip(parts, parts[1:]))
    assert not got


def test_row_tiles_of_a_chunk_go_over_the_same_keys_together():
    """4 row tiles over 586 key tiles on 152 CTAs: CTAs that hold row tiles of one chunk are a few
    keys apart at any time."""
    runs, _ = cut([(2, 586, 4)] * 4, 152)
    for tick in range(0, 120, 7):
        at = {}
        for mine in runs:
            left = tick
            for b, h, row, k0, k1 in mine:
                if left < k1 - k0:
                    at.setdefault((b, h), []).append(k0 + left)
                    break
                left -= k1 - k0
        for keys in at.values():
            keys.sort()
            near = sum(any(j != i and abs(k - keys[j]) <= 20 for j in range(len(keys))) for i, k in enumerate(keys))
            assert near >= 0.8 * len(keys)

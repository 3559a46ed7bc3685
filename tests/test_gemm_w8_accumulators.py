"""Host model of the 8-bit product's second kernel from its stages to its epilogue
(csrc/gemm_w8.cu), run under random interleavings of its roles: the rings as in
test_gemm_w8_protocol.py (256 tokens with the two converter groups they have), and with them the
accumulators, which a CTA's tiles take in turn.

Per tile (KB k-blocks, counted on through all of a CTA's tiles): issuer i of I takes the k-blocks
that are i modulo I of all the CTA's, after the epilogue has emptied the accumulator's buffer
(tile % ACC, acc_empty counts the epilogue's warps), each into an accumulator of its own; when
its last one of the tile is issued it commits to acc_full (which counts the issuers, also one
without a k-block in the tile). The epilogue's warps wait for acc_full, take the sums and
arrive on acc_empty. A tile of one k-block is in one issuer's accumulator only: the one that the
tile's number names. The model holds that every accumulator read by the epilogue holds exactly its
tile's k-blocks, and that no accumulator is written while it is read.
"""
import random

import pytest

from test_pipeline_protocol import Barrier

SHAPES = {64: dict(SQ=4, SA=4, SB=6, BS=1, G=4, I=2, ACC=2), 128: dict(SQ=4, SA=4, SB=4, BS=1, G=4, I=1, ACC=2),
          256: dict(SQ=4, SA=4, SB=5, BS=2, G=2, I=1, ACC=1)}


def run(KB, tiles, seed, SQ, SA, SB, BS, G, I, ACC, epilogue_warps=8, empties=None, single=lambda tile: tile & 1):
    SD, n = max(SA, SB), KB * tiles
    q_full, q_empty = [Barrier(1) for _ in range(SQ)], [Barrier(4) for _ in range(SQ)]
    a_full, b_full, done = [Barrier(4) for _ in range(SA)], [Barrier(1) for _ in range(SB)], [Barrier(1) for _ in range(SD)]
    acc_full, acc_empty = [Barrier(I) for _ in range(ACC)], [Barrier(empties or epilogue_warps) for _ in range(ACC)]
    q, a, b = [None] * SQ, [None] * SA, [None] * SB
    acc = [[[] for _ in range(I)] for _ in range(ACC)]  # k-blocks summed, by buffer and issuer
    rng = random.Random(seed)
    pos = dict(w=0, t=0)
    conv = [[g, 0] for g in range(G) for _ in range(4)]  # each warp's next k-block; has it let go of the codes
    issue = [dict(tile=0, kb=i, stage=0, waited=False) for i in range(I)]  # kb: in the tile
    epi = [0] * epilogue_warps

    def finished(i):
        return i < 0 or done[i % SD].test(i // SD)

    def weights():
        i = pos["w"]
        if i >= n or (i >= SQ and not q_empty[i % SQ].test(i // SQ - 1)):
            return False
        q[i % SQ] = i
        q_full[i % SQ].arrive(i // SQ)
        pos["w"] += 1
        return True

    def convert(w):
        i, _ = conv[w]
        if i >= n or not q_full[i % SQ].test(i // SQ) or not finished(i - SA):
            return False
        assert q[i % SQ] == i
        a[i % SA] = i
        q_empty[i % SQ].arrive(i // SQ)
        a_full[i % SA].arrive(i // SA)
        conv[w][0] += G
        return True

    def tokens():
        j = pos["t"]
        if j >= n * BS or (j >= SB and not finished((j - SB) // BS)):
            return False
        b[j % SB] = j
        b_full[j % SB].arrive(j // SB)
        pos["t"] += 1
        return True

    def mma(me):
        s = issue[me]
        if s["tile"] >= tiles:
            return False
        buf, turn = s["tile"] % ACC, s["tile"] // ACC
        if not s["waited"]:
            if turn > 0 and not acc_empty[buf].test(turn - 1):
                return False
            s["waited"] = True
            acc[buf][me] = [] if s["kb"] < KB else acc[buf][me]  # (the first product does not accumulate)
            return True
        if s["kb"] >= KB:  # the tile's end
            acc_full[buf].arrive(turn)
            s.update(tile=s["tile"] + 1, kb=s["kb"] - KB, stage=0, waited=False)
            return True
        i = s["tile"] * KB + s["kb"]
        j = i * BS + s["stage"]
        if not a_full[i % SA].test(i // SA) or not b_full[j % SB].test(j // SB):
            return False
        assert a[i % SA] == i and b[j % SB] == j
        s["stage"] += 1
        if s["stage"] == BS:
            acc[buf][me].append(i)
            done[i % SD].arrive(i // SD)
            s.update(kb=s["kb"] + I, stage=0)
        return True

    def epilogue(w):
        t = epi[w]
        if t >= tiles or not acc_full[t % ACC].test(t // ACC):
            return False
        got = acc[t % ACC]
        got = got[single(t) if I == 2 else 0] if KB == 1 else sorted(sum(got, []))
        assert got == list(range(t * KB, (t + 1) * KB)), f"warp {w} reads {got} in tile {t}"
        acc_empty[t % ACC].arrive(t // ACC)
        epi[w] += 1
        return True

    roles = ([weights, tokens] + [lambda w=w: convert(w) for w in range(4 * G)] + [lambda m=m: mma(m) for m in range(I)]
             + [lambda w=w: epilogue(w) for w in range(epilogue_warps)])
    idle = 0
    while any(t < tiles for t in epi):
        idle = 0 if rng.choice(roles)() else idle + 1
        assert idle < 20000, f"no role can move: {pos} {conv} {issue} {epi}"
    # the issuers end where all k-blocks are issued
    assert all(s["tile"] == tiles for s in issue) or I == 1 and issue[0]["tile"] == tiles


@pytest.mark.parametrize("BN", [64, 128, 256])
@pytest.mark.parametrize("KB,tiles", [(1, 1), (1, 2), (1, 9), (2, 7), (3, 7), (4, 5), (5, 6), (16, 4), (33, 3)])
def test_accumulators_hold_under_random_schedules(BN, KB, tiles):
    for seed in range(12):
        run(KB, tiles, seed, **SHAPES[BN])


def test_the_model_catches_an_accumulator_emptied_early():
    """One arrival less on acc_empty: the next tile is written while a warp still reads."""
    with pytest.raises(AssertionError):
        for seed in range(60):
            run(2, 12, seed, **SHAPES[64], empties=7)


def test_the_model_catches_the_other_issuers_accumulator():
    """Tiles of one k-block read from the accumulator of the issuer that had none."""
    with pytest.raises(AssertionError):
        run(1, 4, 0, **SHAPES[64], single=lambda tile: 1 - (tile & 1))

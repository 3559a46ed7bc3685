"""Host model of the 8-bit product's stage barriers (csrc/gemm_w8.cu, more than 32
tokens), run under random interleavings of its roles.

Per k-block i: the weight stream fills packed stage i % SQ once its converters let go
of it; converter group i % G reads the packed stage, waits for the MMAs of k-block i - SA
and fills operand stage i % SA; the token stream fills stage j % SB (a k-block has BS of
them) once the MMAs of the k-block that used it are done; the MMA thread waits for the
operand and token stages and commits to done[i % SD]; with I issuing threads, thread
i % I does.

As an mbarrier tells phases apart by parity alone, a wait for phase n is right only while
the barrier has completed n or n + 1 phases; Barrier checks that, and that every arrival
lands in its own phase.
"""
import random

import pytest

from test_pipeline_protocol import Barrier


def run(SQ, SA, SB, BS, G, n, seed, I=1):
    SD = max(SA, SB)
    q_full, q_empty = [Barrier(1) for _ in range(SQ)], [Barrier(1) for _ in range(SQ)]
    a_full, b_full, done = [Barrier(1) for _ in range(SA)], [Barrier(1) for _ in range(SB)], [Barrier(1) for _ in range(SD)]
    q, a, b = [None] * SQ, [None] * SA, [None] * SB
    rng = random.Random(seed)
    pos = dict(w=0, t=0)
    conv = list(range(G))  # the next k-block of each group
    issue = [[i, 0] for i in range(I)]  # each issuer's next k-block and its token stage

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

    def convert(g):
        i = conv[g]
        if i >= n or not q_full[i % SQ].test(i // SQ) or not finished(i - SA):
            return False
        assert q[i % SQ] == i, f"group {g} read k-block {q[i % SQ]} for {i}"
        a[i % SA] = i
        q_empty[i % SQ].arrive(i // SQ)
        a_full[i % SA].arrive(i // SA)
        conv[g] += G
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
        i, stage = issue[me]
        if i >= n or not a_full[i % SA].test(i // SA):
            return False
        j = i * BS + stage
        if not b_full[j % SB].test(j // SB):
            return False
        assert a[i % SA] == i and b[j % SB] == j
        issue[me][1] += 1
        if stage + 1 == BS:
            done[i % SD].arrive(i // SD)
            issue[me] = [i + I, 0]
        return True

    roles = [weights, tokens] + [lambda g=g: convert(g) for g in range(G)] + [lambda m=m: mma(m) for m in range(I)]
    idle = 0
    while any(i < n for i, _ in issue):
        idle = 0 if rng.choice(roles)() else idle + 1
        assert idle < 10000, f"no role can move: {pos} {conv} {issue}"


@pytest.mark.parametrize("SQ,SA,SB,BS,G,I", [(4, 4, 6, 1, 4, 2), (4, 4, 4, 1, 4, 1), (4, 4, 5, 2, 4, 1)])
def test_rings_hold_under_random_schedules(SQ, SA, SB, BS, G, I):
    for seed in range(40):
        run(SQ, SA, SB, BS, G, 83, seed, I)


def test_the_model_catches_fewer_packed_stages_than_groups():
    """A group then waits on a barrier two phases behind, whose parity looks complete."""
    with pytest.raises(AssertionError):
        for seed in range(40):
            run(2, 4, 3, 1, 4, 83, seed)

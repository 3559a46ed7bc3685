"""Host model of the tensor-memory attention's barriers (csrc/prefix_tc.cu), run under random
interleavings of its roles.

K and V tiles pass through one ring of slots in the order K0 K1 V0 K2 V1 ... V(n-1). One
thread issues the scores' products (K tiles, two score buffers), one the outputs' (V tiles),
and the softmax warps turn a tile's scores into weights (two buffers); now and then they
rescale the output, for which the product before has to be complete. An mbarrier tells phases
apart by parity alone: Barrier checks that every wait is for the phase at hand or the one
before, and every arrival in its own phase.
"""
import random

import pytest

from test_pipeline_protocol import Barrier


def order(n):
    seq = [("K", 0)]
    for i in range(n):
        if i + 1 < n:
            seq.append(("K", i + 1))
        seq.append(("V", i))
    return seq


def run(NS, n, seed, wait_weights_free=True):
    rng = random.Random(seed)
    seq = order(n)
    at = {x: pos for pos, x in enumerate(seq)}
    full, empty = [Barrier(1) for _ in range(NS)], [Barrier(1) for _ in range(NS)]
    s_full, p_full, pv_done = ([Barrier(1) for _ in range(2)] for _ in range(3))
    slot, scores, weights = [None] * NS, [None, None], [None, None]
    pos = dict(load=0, qk=0, pv=0, soft=0)
    done_pv = -1

    def load():
        p = pos["load"]
        if p >= len(seq) or (p >= NS and not empty[p % NS].test(p // NS - 1)):
            return False
        slot[p % NS] = seq[p]
        full[p % NS].arrive(p // NS)
        pos["load"] += 1
        return True

    def qk():
        i = pos["qk"]
        if i >= n:
            return False
        p = at["K", i]
        if (i >= 2 and not p_full[i & 1].test((i - 2) // 2)) or not full[p % NS].test(p // NS):
            return False
        assert slot[p % NS] == ("K", i) and (i < 2 or pos["soft"] > i - 2)
        scores[i & 1] = i
        empty[p % NS].arrive(p // NS)
        s_full[i & 1].arrive(i // 2)
        pos["qk"] += 1
        return True

    def pv():
        nonlocal done_pv
        i = pos["pv"]
        if i >= n:
            return False
        p = at["V", i]
        if not full[p % NS].test(p // NS) or not p_full[i & 1].test(i // 2):
            return False
        assert slot[p % NS] == ("V", i) and weights[i & 1] == i
        empty[p % NS].arrive(p // NS)
        done_pv = i
        pv_done[i & 1].arrive(i // 2)
        pos["pv"] += 1
        return True

    rescales = [rng.random() < 0.3 for _ in range(n)]

    def soft():
        i = pos["soft"]
        if i >= n or not s_full[i & 1].test(i // 2):
            return False
        assert scores[i & 1] == i
        if i > 0 and rescales[i]:
            if not pv_done[(i - 1) & 1].test((i - 1) // 2):
                return False
            assert done_pv == i - 1
        if wait_weights_free and i >= 2 and not pv_done[i & 1].test((i - 2) // 2):
            return False
        assert i < 2 or done_pv >= i - 2, "weights overwritten before their product"
        weights[i & 1] = i
        p_full[i & 1].arrive(i // 2)
        pos["soft"] += 1
        return True

    roles, idle = [load, qk, pv, soft], 0
    while pos["pv"] < n:
        idle = 0 if rng.choice(roles)() else idle + 1
        assert idle < 10000, f"no role can move: {pos}"
    assert pv_done[(n - 1) & 1].test((n - 1) // 2)


@pytest.mark.parametrize("NS", [5, 6, 8])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 7, 50, 51])
def test_barriers_hold_under_random_schedules(NS, n):
    for seed in range(40):
        run(NS, n, seed)


def test_the_model_catches_weights_overwritten_early():
    with pytest.raises(AssertionError):
        for seed in range(60):
            run(6, 60, seed, wait_weights_free=False)

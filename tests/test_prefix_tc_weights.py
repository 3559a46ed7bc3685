"""The tensor-memory attention's softmax weights (csrc/prefix_tc.cu): two bf16 parts, written
over the scores that they came from.

Precision: a weight's two parts hold it within 2^-16, and fp32 scores and exponentials move it
by about 1e-5 here, so an output differs from the correctly rounded one only where it lies that
near to a rounding border. Hence (a) where every position's value is the same power of two
the output is that value exactly, as its weights sum to one within 2^-15 and bf16's nearest
neighbours are 2^-8 away, and (b) the error's 2-norm is the output rounding's own, taken from the
64-bit result itself, with a tenth more for the rest. (One bf16 part has 1.4 times that norm.)

Host model of the columns' hand-over: scores of tile i + NB go where the weights of tile i were
once their product is complete. Roles and Barrier as in test_prefix_tc_protocol.py, whose
columns of weights were apart from the scores'.
"""
import random

import pytest

from test_pipeline_protocol import Barrier

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


def tensor_memory(B, P, S, Hq, Hkv, d):
    """Whether the sizes go to the tensor-memory kernel: a workspace for partial states, more
    than 32 query rows a KV head, 256 shared positions."""
    from bit_moe_expert_route_gb300 import ops
    n = ops.lib().moe_prefix_attention_workspace_bytes(B, P, S, Hq, Hkv, d)
    return n > 256 and B * (Hq // Hkv) > 32 and P >= 256


@gpu
@pytest.mark.parametrize("B,P,S,Hq,Hkv,d", [(64, 5000, 9, 16, 2, 256), (60, 3000, 0, 12, 4, 128), (70, 2500, 33, 8, 8, 64),
                                            (33, 2500, 0, 16, 1, 256)])
def test_error_is_the_output_rounding(B, P, S, Hq, Hkv, d):
    import test_prefix_attention as A
    from bit_moe_expert_route_gb300 import ops
    assert tensor_memory(B, P, S, Hq, Hkv, d)
    x = A.inputs(B, P, S, Hq, Hkv, d, 3)
    o, _ = A.expected(*x)
    own = (o.to(torch.bfloat16).double() - o).norm()
    assert float((ops.prefix_attention(*x).double() - o).norm()) <= 1.1 * float(own)


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_weights_sum_to_one(d):
    """Rows with one, two or a few dominant positions and rows of even ones, in slices of many
    tiles (their reference is an earlier score than the largest); the values are a power of
    two for each element, the same at every position."""
    import test_prefix_attention as A
    from bit_moe_expert_route_gb300 import ops
    B, P, S = 600, 4100, 20
    assert tensor_memory(B, P, S, 16, 16, d)
    q, kp, vp, ks, vs, ln = A.inputs(B, P, S, 16, 16, d, 9)
    q *= torch.tensor([0.1, 1.0, 2.0, 2.5, 3.0, 4.0], device="cuda").bfloat16().repeat(B // 6)[:, None, None]
    v = torch.exp2(torch.arange(16 * d, device="cuda") % 9 - 4).view(16, d).bfloat16()
    vp[:], vs[:] = v, v
    got = ops.prefix_attention(q, kp, vp, ks, vs, ln)
    assert torch.equal(got, v.expand(B, 16, d))


def order(n):
    seq = [("K", 0)]
    for i in range(n):
        if i + 1 < n:
            seq.append(("K", i + 1))
        seq.append(("V", i))
    return seq


def run(NS, n, seed, scores_wait_for="product", NB=3):
    rng = random.Random(seed)
    seq = order(n)
    at = {x: pos for pos, x in enumerate(seq)}
    full, empty = [Barrier(1) for _ in range(NS)], [Barrier(1) for _ in range(NS)]
    s_full, pv_done = ([Barrier(1) for _ in range(NB)] for _ in range(2))
    p_full = [Barrier(4) for _ in range(NB)]
    slot = [None] * NS
    columns = [[None] * 4 for _ in range(NB)]  # a buffer's content for each warp's lanes: ("scores" | "weights", tile)
    pos = dict(load=0, qk=0, pv=0)
    soft = [0] * 4
    rescales = [[rng.random() < 0.3 for _ in range(n)] for _ in range(4)]

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
        free = pv_done if scores_wait_for == "product" else p_full
        p = at["K", i]
        if (i >= NB and not free[i % NB].test((i - NB) // NB)) or not full[p % NS].test(p // NS):
            return False
        assert slot[p % NS] == ("K", i)
        assert i < NB or pos["pv"] > i - NB, "weights overwritten before their product"
        columns[i % NB] = [("scores", i)] * 4
        empty[p % NS].arrive(p // NS)
        s_full[i % NB].arrive(i // NB)
        pos["qk"] += 1
        return True

    def pv():
        i = pos["pv"]
        if i >= n:
            return False
        p = at["V", i]
        if not full[p % NS].test(p // NS) or not p_full[i % NB].test(i // NB):
            return False
        assert slot[p % NS] == ("V", i) and columns[i % NB] == [("weights", i)] * 4
        empty[p % NS].arrive(p // NS)
        pos["pv"] += 1
        pv_done[i % NB].arrive(i // NB)
        return True

    def softmax(w):
        i = soft[w]
        if i >= n or not s_full[i % NB].test(i // NB):
            return False
        assert columns[i % NB][w] == ("scores", i)
        if i > 0 and rescales[w][i]:
            if not pv_done[(i - 1) % NB].test((i - 1) // NB):
                return False
            assert pos["pv"] == i  # the output is whole, and the next product has not begun
        columns[i % NB][w] = ("weights", i)
        p_full[i % NB].arrive(i // NB)
        soft[w] += 1
        return True

    roles, idle = [load, qk, pv] + [lambda w=w: softmax(w) for w in range(4)], 0
    while pos["pv"] < n:
        idle = 0 if rng.choice(roles)() else idle + 1
        assert idle < 10000, f"no role can move: {pos} {soft}"
    assert pv_done[(n - 1) % NB].test((n - 1) // NB)


@pytest.mark.parametrize("NS", [5, 6, 8])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 7, 50, 51])
def test_columns_hold_under_random_schedules(NS, n):
    for seed in range(40):
        run(NS, n, seed)


def test_the_model_catches_scores_over_unused_weights():
    with pytest.raises(AssertionError):
        for seed in range(60):
            run(6, 60, seed, scores_wait_for="weights")

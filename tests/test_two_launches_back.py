"""Grids that run beside their predecessor (the 8-bit product's weight stream beside the widening
kernel, the own positions beside the tensor-memory attention) and read what was written
before that predecessor: the chain of synchronisation that makes it visible.

Host model, under random schedules: run r writes its data (P), then grid A waits for it,
triggers its dependents and releases the call's ticket; blocks of grid B start once all of A's
blocks have triggered, poll the ticket's word and take what the releasing thread saw, or wait
for A's end; the call's last kernel clears the word. A graph runs again with the same ticket.
Each block has to see its own run's data.

On the GPU: graphs whose first nodes write the data anew each time they run.
"""
import random

import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


def run(seed, runs=6, blocks=4, polls=3, same_ticket=True, clears=True, acquires=True, b_clears=False):
    rng = random.Random(seed)
    word = dict(ticket=rng.choice([0, 12345]), sees=-1)  # a workspace is not initialised
    for r in range(runs):
        ticket = 77 if same_ticket else 77 + r
        triggered, released, a_done = 0, False, False
        state = ["idle"] * blocks  # of B: idle, polling, waiting, read
        polled, view = [0] * blocks, [-1] * blocks
        while "read" not in state or set(state) != {"read"} or not a_done:
            move = rng.randrange(blocks + 3)
            if move == 0 and triggered < blocks:
                triggered += 1  # (that block of A has waited: it sees run r)
            elif move == 1 and triggered > 0 and not released:
                word.update(ticket=ticket, sees=r)
                released = True
            elif move == 2 and triggered == blocks and released and rng.random() < 0.2:
                a_done = True
            elif move >= 3 and triggered == blocks:
                b = move - 3
                if state[b] == "idle":
                    state[b] = "polling" if acquires else "read"
                elif state[b] == "polling":
                    polled[b] += 1
                    if word["ticket"] == ticket:
                        view[b], state[b] = word["sees"], "read"
                    elif polled[b] == polls:
                        state[b] = "waiting"
                elif state[b] == "waiting" and a_done:
                    view[b], state[b] = r, "read"
                if state[b] == "read":
                    assert view[b] == r, f"run {r}: block {b} sees run {view[b]}"
                    if b_clears and b == 0 and a_done:  # the product's first block, at its end
                        word.update(ticket=0, sees=-1)
        if clears:
            word.update(ticket=0, sees=-1)


@pytest.mark.parametrize("same_ticket", [True, False])
@pytest.mark.parametrize("b_clears", [True, False])
def test_every_block_sees_its_own_run(same_ticket, b_clears):
    for seed in range(300):
        run(seed, same_ticket=same_ticket, b_clears=b_clears)


def test_the_model_catches_a_ticket_that_stays():
    with pytest.raises(AssertionError):
        for seed in range(300):
            run(seed, clears=False)


def test_the_model_catches_reading_without_the_ticket():
    with pytest.raises(AssertionError):
        run(0, acquires=False)


def replays(write, call, fresh):
    """A graph of `write` (from staging tensors) and `call`, run with new contents each time."""
    write(), call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        write()
        out = call()
        write()
        again = call()
    for i in range(8):
        want = fresh(i)
        out.zero_(), again.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(again, want), i


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_own_positions_written_just_before(d):
    import test_prefix_attention as A
    from bit_moe_expert_route_gb300 import ops
    B, P, S, Hq, Hkv = 40, 700, 90, 8, 2
    n = ops.lib().moe_prefix_attention_workspace_bytes(B, P, S, Hq, Hkv, d)
    assert n > 256  # not the one launch of clusters
    q, kp, vp, ks, vs, ln = A.inputs(B, P, S, Hq, Hkv, d, 1)
    stage = [t.clone() for t in (q, ks, vs, ln)]
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def write():
        for t, s in zip((q, ks, vs, ln), stage):
            t.copy_(s)

    def fresh(i):
        x = A.inputs(B, P, S, Hq, Hkv, d, 100 + i)
        for s, t in zip(stage, (x[0], x[3], x[4], x[5])):
            s.copy_(t)
        return ops.prefix_attention(x[0], kp, vp, x[3], x[4], x[5])
    replays(write, lambda: ops.prefix_attention(q, kp, vp, ks, vs, ln, ws=ws), fresh)


@gpu
@pytest.mark.parametrize("T,N,K", [(40, 20000, 64), (64, 20000, 512), (100, 20000, 256), (300, 40000, 2048)])
def test_weights_written_just_before(T, N, K):
    import test_gemm_w8a8 as W
    from bit_moe_expert_route_gb300 import ops
    n = ops.lib().moe_gemm_w8a8_workspace_bytes(T, N, K)
    assert n > 256  # the tensor-memory kernel
    x = W.inputs(T, N, K, 1)
    stage = [t.clone() for t in x]
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def write():
        for t, s in zip(x, stage):
            t.copy_(s)

    def fresh(i):
        y = W.inputs(T, N, K, 100 + i)
        for s, t in zip(stage, y):
            s.copy_(t)
        return ops.gemm_w8a8(*y)
    replays(write, lambda: ops.gemm_w8a8(*x, ws=ws), fresh)

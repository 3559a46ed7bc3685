"""examples/score_continuations.py: a step that the caches have no room for is refused on the host
(its keys would be written past the cache's end)."""
import os
import sys

import pytest

pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_no_room():
    from score_continuations import Continuations
    c = Continuations.__new__(Continuations)  # (no weights: the refusal comes first)
    c.room = c.steps = 3
    with pytest.raises(ValueError, match="3 positions"):
        c.step(None, None)


@pytest.mark.gpu
def test_room_steps_are_taken():
    import torch
    from bit_moe_expert_route_gb300.synth import LayerShape
    from score_continuations import Continuations
    c = Continuations(2, 70, room=2, vocab=1000, shape=LayerShape(d_model=256, n_experts=32, top_k=4, d_ff=256, d_ff_shared=256),
                      heads=(16, 2, 64))
    t = torch.arange(2, dtype=torch.int32, device="cuda")
    for _ in range(2):
        c.step(t, t)
    with pytest.raises(ValueError, match="2 positions"):
        c.step(t, t)
    assert c.lens.tolist() == [2, 2]

"""examples/score_continuations.py: every stage of a step against its own formula on the
values that the stage before gave it, with the tolerances of the operators' tests."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("batch,prompt", [(1, 70), (5, 700), (40, 300)])
def test_stages_of_a_step(batch, prompt):
    import test_gemm_w8a8 as G
    import test_logprob as P
    import test_norm_q8 as N
    import test_prefix_attention as A
    from bit_moe_expert_route_gb300.synth import LayerShape
    from score_continuations import Continuations
    def near(got, ref):  # bf16 outputs: fp32 scales (1.3e-7) and one rounding, half a step at most
        assert torch.all((got.double() - ref).abs() <= (2.0 ** -8 + 2e-7) * ref.abs())
    shape = LayerShape(d_model=256, n_experts=32, top_k=4, d_ff=256, d_ff_shared=256)
    c = Continuations(batch, prompt, room=3, vocab=1000, shape=shape, heads=(16, 2, 64))
    tokens = torch.arange(batch, dtype=torch.int32, device="cuda")
    for i in range(3):
        wanted = (tokens + 17 * i) % 1000
        r = c.step(tokens, wanted)
        N.check(r["x"], None, c.norms[0], "int8", r["n1"])
        near(r["qkv"], G.exact(r["n1"].q, r["n1"].scale, *c.w_qkv))
        q = r["qkv"].view(batch, 20, 64)[:, :16].contiguous()
        assert torch.equal(c.k_own[:, i], r["qkv"].view(batch, 20, 64)[:, 16:18])
        assert torch.all(c.lens == i + 1)
        A.check(r["att"], *A.expected(q, c.k_prompt, c.v_prompt, c.k_own, c.v_own, c.lens))
        N.check(r["att"].view(batch, -1), None, c.norms[1], "int8", r["n2"])
        near(r["out"], G.exact(r["n2"].q, r["n2"].scale, *c.w_out))
        N.check(r["out"], r["n1"].residual, c.norms[2], "int8", r["n3"])
        assert torch.isfinite(r["moe"]).all() and r["moe"].shape == (batch, 256)
        N.check(r["moe"], r["n3"].residual, c.norms[3], "int8", r["n4"])
        ref = G.exact(r["n4"].q, r["n4"].scale, *c.w_head)
        assert torch.all((r["logits"].double() - ref).abs() <= 1.3e-7 * ref.abs())
        P.check(r["logits"], wanted, 5, r["scores"])
        tokens = r["scores"].top_ids[:, 0].contiguous()

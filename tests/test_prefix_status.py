"""The status word of moe_prefix_attention's workspace: every call that has one clears it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,P,S,Hq,Hkv,d", [
    (400, 0, 0, 4, 2, 64), (400, 0, 0, 4, 2, 256), (1, 0, 0, 1024, 1024, 64),  # nothing to attend to, too many blocks for one launch
    (2, 0, 0, 4, 2, 64), (2, 700, 16, 16, 2, 256),                           # one launch
    (400, 0, 20, 4, 2, 64), (400, 90, 0, 4, 2, 64), (400, 90, 20, 4, 2, 64),  # warps' products
    (64, 3000, 0, 16, 2, 128), (64, 3000, 20, 16, 2, 128)])                   # tensor memory
def test_every_call_clears_the_status(B, P, S, Hq, Hkv, d):
    import test_prefix_attention as A
    from bit_moe_expert_route_gb300 import ops
    x = A.inputs(B, P, S, Hq, Hkv, d, 1)
    n = ops.lib().moe_prefix_attention_workspace_bytes(B, P, S, Hq, Hkv, d)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    got = ops.prefix_attention(*x, ws=ws)
    assert ops.device_status(ws) == 0
    assert torch.equal(got, ops.prefix_attention(*x)) and (P + S > 0 or not got.any())

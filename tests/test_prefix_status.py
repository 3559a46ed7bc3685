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


@pytest.mark.parametrize("B,P,S", [(3, 400, 20), (40, 20, 300), (6, 3000, 20), (40, 700, 20)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_infinite_scores(B, P, S, d):
    """One launch, warps' products and tensor memory: a row whose every score is -infinity is
    zeros, one with a score of +infinity is NaN, others are as they were."""
    import test_prefix_attention as A
    from bit_moe_expert_route_gb300 import ops
    q, kp, vp, ks, vs, ln = A.inputs(B, P, S, 8, 2, d, d, [S] * B)
    q[:, :, 0] = q[:, :, 0].abs() + 0.5  # every score of KV head 0 is -infinity ...
    kp[:, 0, 0], ks[:, :, 0, 0] = -float("inf"), -float("inf")
    kp[P - 1, 1, 1] = float("inf")       # ... and one of head 1 is +infinity where q is positive, -infinity where not
    q[:, 4:, 1] = torch.where(torch.arange(4, device="cuda") % 2 == 0, 1.0, -1.0).bfloat16()
    got = ops.prefix_attention(q, kp, vp, ks, vs, ln)
    assert not got[:, :4].any()
    assert torch.isnan(got[:, 4::2]).all()
    o, mag = A.expected(q, kp, vp, ks, vs, ln)
    A.check(got[:, 5::2], o[:, 5::2], mag[:, 5::2])

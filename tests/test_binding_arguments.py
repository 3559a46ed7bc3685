"""Arguments of the operators around the layer that the binding has to take or to refuse."""
import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@gpu
def test_strides_of_axes_of_one_entry_do_not_count():
    """K and V of one position, one KV head or one sequence, whose strides differ only there."""
    import test_prefix_attention as A
    from bit_moe_expert_route_gb300 import ops
    for B, P, S, Hkv in ((1, 1, 1, 2), (1, 300, 30, 1), (3, 1, 20, 2), (3, 50, 1, 1), (40, 300, 1, 1)):
        q, kp, vp, ks, vs, ln = A.inputs(B, P, S, 4 * Hkv, Hkv, 64, 3, [S] * B)

        def odd(t):  # the same values, with other strides on its axes of one entry
            return t.as_strided(t.shape, [24 * st + 8 if n == 1 and i < t.dim() - 1 else st
                                          for i, (n, st) in enumerate(zip(t.shape, t.stride()))])
        want = ops.prefix_attention(q, kp, vp, ks, vs, ln)
        assert odd(vp).stride() != vp.stride() or odd(vs).stride() != vs.stride()
        assert torch.equal(ops.prefix_attention(q, kp, odd(vp), ks, odd(vs), ln), want)
        assert torch.equal(ops.prefix_attention(q, odd(kp), vp, odd(ks), vs, ln), want)
        A.check(want, *A.expected(q, kp, vp, ks, vs, ln))


def test_values_without_keys():
    from bit_moe_expert_route_gb300 import ops
    q, k = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_suffix"):
        ops.prefix_attention(q, k, k, v_suffix=torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16))


@gpu
def test_workspaces_that_no_kernel_can_use():
    """Host memory, and views with gaps, are refused before anything is enqueued; a workspace of
    another type counts in bytes."""
    import test_gemm_w8a8 as W
    import test_prefix_attention as A
    from bit_moe_expert_route_gb300 import ops
    x, y = W.inputs(40, 20000, 64, 1), A.inputs(4, 3000, 20, 16, 2, 64, 1)
    n = ops.lib().moe_gemm_w8a8_workspace_bytes(40, 20000, 64)
    m = ops.lib().moe_prefix_attention_workspace_bytes(4, 3000, 20, 16, 2, 64)
    for call, size in ((lambda ws: ops.gemm_w8a8(*x, ws=ws), n), (lambda ws: ops.prefix_attention(*y, ws=ws), m)):
        for ws in (torch.empty(size, dtype=torch.uint8), torch.empty(2 * size, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError, match="ws"):
                call(ws)
        with pytest.raises(ops.MoeError):
            call(torch.empty(size - 1, dtype=torch.uint8, device="cuda"))
        assert torch.equal(call(torch.empty(size // 4 + 1, dtype=torch.int32, device="cuda")),
                           call(torch.empty(size, dtype=torch.uint8, device="cuda")))

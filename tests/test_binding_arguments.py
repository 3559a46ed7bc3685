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

"""Every kernel of the 8-bit product and the shared-prefix attention on the inputs where it can
go wrong: all codes, sums past 2^24, single k-blocks, NaN scales, strided outputs, far rows;
stale and clamped positions, graphs whose lengths change. A case names the kernel that it is
for, and a test on a runtime that launches nothing (fake_cuda.py) holds that it goes there.
Tolerances and references are those of test_gemm_w8a8 and test_prefix_attention.
"""
import shutil

import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu

KS = [16, 64, 128, 144, 8192]  # less than a k-block, whole and ragged ones, sums past 2^24
PRODUCTS = [(kernel, T, N, K) for kernel, T, N, ks in (
    ("gemm_w8_few_kernel<1, 1>", 5, 300, KS), ("gemm_w8_few_kernel<1, 2>", 16, 300, KS), ("gemm_w8_few_kernel<1, 3>", 24, 300, KS),
    ("gemm_w8_few_kernel<1, 4>", 70, 300, KS), ("gemm_w8_few_kernel<2, 1>", 8, 20011, KS), ("gemm_w8_few_kernel<2, 2>", 13, 20011, KS),
    ("gemm_w8_few_kernel<2, 3>", 24, 20011, KS), ("gemm_w8_kernel<64, false>", 40, 20011, KS), ("gemm_w8_kernel<64, false>", 64, 40000, KS),
    ("gemm_w8_kernel<128, false>", 100, 20011, KS), ("gemm_w8_kernel<128, false>", 300, 40000, KS[:4]),
    ("gemm_w8_kernel<256, false>", 4097, 20011, KS[:4]), ("gemm_w8_kernel<256, false>", 300, 40000, KS[4:])) for K in ks]

PREFIX = [("prefix_joined_kernel", 8, 70, 130, 8, 2), ("prefix_joined_kernel", 3, 0, 130, 16, 1), ("prefix_kernel<D, 1>", 16, 70, 130, 8, 8),
          ("prefix_kernel<D, 1>", 4, 3000, 130, 4, 2), ("prefix_kernel<D, 2>", 8, 3000, 130, 8, 2), ("prefix_kernel<D, 2>", 48, 0, 130, 8, 2),
          ("prefix_tc_kernel", 40, 300, 130, 8, 2), ("prefix_tc_kernel", 48, 2500, 130, 16, 4)]


PREFIXES = [(kernel.replace("<D", f"<{d}") if "<D" in kernel else f"{kernel}<{d}>", *shape, d)
            for kernel, *shape in PREFIX for d in (64, 128, 256)]


@pytest.mark.skipif(not shutil.which("g++"), reason="the fake runtime needs g++")
def test_cases_go_to_their_kernels():
    import fake_cuda as F
    L = F.lib()
    for kernel, T, N, K in PRODUCTS:
        L.fake_reset()
        assert F.gemm(L, T, N, K) == 0
        names = [n for n, *_ in F.launches(L)]
        assert names == ([kernel] if "few" in kernel else ["widen_kernel", kernel]), (T, N, K)
    for kernel, *shape in PREFIXES:
        L.fake_reset()
        assert F.prefix(L, *shape) == 0
        names = [n for n, *_ in F.launches(L)]
        assert kernel in names, (kernel, shape, names)
        if "tc" in kernel:
            assert [n.split("<")[0] for n in names] == ["prefix_tc_kernel", "prefix_kernel", "prefix_combine_kernel"]


@gpu
@pytest.mark.parametrize("kernel,T,N,K", PRODUCTS)
def test_every_code(kernel, T, N, K):
    """All 256 codes with rows of nothing but -128 and 127; one token's scale is NaN; an output
    with gaps between its rows."""
    import test_gemm_w8a8 as W
    from bit_moe_expert_route_gb300 import ops
    a, sa, w, sw = W.inputs(T, N, K, T + N + K, extreme=True)
    a[0], w[0], w[1] = -128, -128, 127
    a[1], w[2, ::2], w[2, 1::2] = 127, -128, 127
    w[N - 1] = -128
    ref = W.exact(a, sa, w, sw)
    bound = 1.3e-7 * ref.abs()
    if K > 1024:
        bound = bound + K / 16 * 2.0 ** -23 * W.exact(a.double().abs(), sa, w.double().abs(), sw)
    got = ops.gemm_w8a8(a, sa, w, sw, dtype=torch.float32)
    assert torch.all((got.double() - ref).abs() <= bound)
    wide = torch.full((T, N + 13), 7.0, device="cuda", dtype=torch.bfloat16)
    sa[T - 1] = float("nan")
    ops.gemm_w8a8(a, sa, w, sw, out=wide[:, 5:N + 5])
    assert torch.equal(wide[:T - 1, 5:N + 5], got[:T - 1].to(torch.bfloat16))
    assert torch.isnan(wide[T - 1, 5:N + 5]).all()
    assert torch.all(wide[:, :5] == 7) and torch.all(wide[:, N + 5:] == 7)


@gpu
@pytest.mark.parametrize("T,N", [(8, 300), (24, 300), (24, 20011)])
def test_far_rows_of_few_tokens(T, N):
    """Rows of tokens and of the output whose offsets pass 2^31 elements."""
    import test_gemm_w8a8 as W
    from bit_moe_expert_route_gb300 import ops
    a, sa, w, sw = W.inputs(T, N, 256, 1)
    ld = (1 << 31) // (T - 1) // 16 * 16 + 32
    far = torch.empty((T - 1) * ld + 256, dtype=torch.int8, device="cuda").as_strided((T, 256), (ld, 1))
    out = torch.empty((T - 1) * ld + N, dtype=torch.bfloat16, device="cuda").as_strided((T, N), (ld, 1))
    assert (T - 1) * ld >= 1 << 31
    far.copy_(a)
    assert torch.equal(ops.gemm_w8a8(far, sa, w, sw, out=out), ops.gemm_w8a8(a, sa, w, sw))
    del far, out
    torch.cuda.empty_cache()


def ragged(B, S):
    return [(0, 1, 63, 64, 65, S, -3, 4000)[i % 8] for i in range(B)]


@gpu
@pytest.mark.parametrize("kernel,B,P,S,Hq,Hkv,d", PREFIXES)
def test_stale_positions_and_changing_lengths(kernel, B, P, S, Hq, Hkv, d):
    """Positions past a sequence's length hold NaN and infinities, lengths are clamped to 0 .. S;
    then the same call in a graph, with other lengths when it runs."""
    import test_prefix_attention as A
    from bit_moe_expert_route_gb300 import ops
    lens = ragged(B, S)
    q, kp, vp, ks, vs, ln = A.inputs(B, P, S, Hq, Hkv, d, d, lens)
    whole = ks.clone(), vs.clone()
    for b, n in enumerate(lens):
        n = min(max(n, 0), S)
        ks[b, n:], vs[b, n:] = float("nan"), float("inf")
    want = ops.prefix_attention(q, kp, vp, ks, vs, ln)
    A.check(want, *A.expected(q, kp, vp, ks, vs, ln))
    out = torch.empty_like(want)
    ws = torch.empty(ops.lib().moe_prefix_attention_workspace_bytes(B, P, S, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.prefix_attention(q, kp, vp, ks, vs, ln, out=out, ws=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    ks.copy_(whole[0]), vs.copy_(whole[1])
    ln.copy_(torch.tensor(ragged(B + 3, S)[3:], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    A.check(out, *A.expected(q, kp, vp, ks, vs, ln))
    assert torch.equal(out, ops.prefix_attention(q, kp, vp, ks, vs, ln)) and not torch.equal(out, want)

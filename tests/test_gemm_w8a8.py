"""moe_gemm_w8a8 against the exact integer product in 64 bits.

fp32 output: the integer sum is exact below 2^24 (every case here that expects
it), then two fp32 multiplications: 2 * 2^-24 relative, so 1.3e-7 bounds it.
Where K is longer and the codes are extreme, the fp32 sum may round once in each of
its K / 16 steps by 2^-24 of its largest partial sum: K / 16 * 2^-24 of the sum of
magnitudes, twice that allowed for truncation in the tensor cores. bf16: 2^-8 more.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


def inputs(T, N, K, seed, pad=0, extreme=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes(rows, ld):
        if extreme:
            return torch.randint(-128, 128, (rows, ld), generator=g, device="cuda").to(torch.int8)
        return torch.randn(rows, ld, generator=g, device="cuda").mul(32).round().clamp(-127, 127).to(torch.int8)
    a = codes(T, K + pad)[:, :K]
    w = codes(N, K)
    return (a, torch.rand(T, generator=g, device="cuda") + 0.5, w, torch.rand(N, generator=g, device="cuda") * 1e-3 + 1e-3)


def exact(a, sa, w, sw):
    return (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()


SHAPES = [(1, 1, 16, 0), (1, 4608, 2048, 0), (2, 100, 48, 16), (7, 333, 2048, 0), (8, 40001, 512, 0), (3, 20480, 16, 0), (31, 30001, 1104, 0), (13, 25000, 8192, 16), (9, 65, 4096, 32), (17, 20011, 272, 0),
          (24, 33, 8192, 0), (32, 2048, 2048, 0), (33, 2048, 2048, 0), (33, 1, 16, 0), (64, 129, 144, 16), (65, 300, 1024, 0), (100, 40000, 256, 0),
          (129, 4608, 2048, 0), (255, 127, 400, 0), (300, 5000, 1040, 0), (700, 8192, 640, 16), (1500, 4100, 2048, 0), (4097, 1029, 528, 0), (4000, 8100, 144, 0),
          (8192, 4100, 1040, 0)]


@gpu
@pytest.mark.parametrize("T,N,K,pad", SHAPES)
def test_exact_sums(T, N, K, pad):
    from bit_moe_expert_route_gb300 import ops
    a, sa, w, sw = inputs(T, N, K, T + N + K, pad)
    ref = exact(a, sa, w, sw)
    ws = torch.empty(ops.lib().moe_gemm_w8a8_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    got = ops.gemm_w8a8(a, sa, w, sw, dtype=torch.float32, ws=ws)
    assert ops.device_status(ws) == 0
    assert torch.all((got.double() - ref).abs() <= 1.3e-7 * ref.abs())
    got16 = ops.gemm_w8a8(a, sa, w, sw, ws=ws)
    assert torch.equal(got16, got.to(torch.bfloat16))
    assert torch.equal(ops.gemm_w8a8(a, sa, w, sw, ws=ws), got16)


@gpu
@pytest.mark.parametrize("T,N,K", [(5, 200, 1024), (40, 200, 1024), (300, 600, 1024), (20, 64, 8192), (200, 300, 8192)])
def test_every_code(T, N, K):
    """All 256 codes, -128 among them; and rows of nothing but -128 and 127."""
    from bit_moe_expert_route_gb300 import ops
    a, sa, w, sw = inputs(T, N, K, K, extreme=True)
    a[0], w[0], w[1] = -128, -128, 127
    a[1, :], w[2, ::2], w[2, 1::2] = 127, -128, 127
    got = ops.gemm_w8a8(a, sa, w, sw, dtype=torch.float32)
    ref = exact(a, sa, w, sw)
    bound = 1.3e-7 * ref.abs()
    if K > 1024:
        bound = bound + K / 16 * 2.0 ** -23 * exact(a.double().abs(), sa, w.double().abs(), sw)
    assert torch.all((got.double() - ref).abs() <= bound)


@gpu
@pytest.mark.parametrize("T", [3, 150])
def test_strided_output_and_other_stream(T):
    from bit_moe_expert_route_gb300 import ops
    a, sa, w, sw = inputs(T, 301, 320, T)
    wide = torch.full((T, 340), 7.0, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ops.gemm_w8a8(a, sa, w, sw, out=wide[:, 5:306])
    s.synchronize()
    assert torch.equal(wide[:, 5:306], exact(a, sa, w, sw).float().to(torch.bfloat16))
    assert torch.all(wide[:, :5] == 7) and torch.all(wide[:, 306:] == 7)
    torch.cuda.synchronize()
    got = ops.gemm_w8a8(a, sa, w, sw, stream=s)  # made on the current stream, used on another
    s.synchronize()
    assert torch.equal(got, wide[:, 5:306])


@gpu
@pytest.mark.parametrize("T", [5, 40, 300])
def test_captured_in_a_graph(T):
    from bit_moe_expert_route_gb300 import ops
    a, sa, w, sw = inputs(T, 4000, 256, T)
    want = ops.gemm_w8a8(a, sa, w, sw)
    out = torch.empty_like(want)
    ws = torch.empty(ops.lib().moe_gemm_w8a8_workspace_bytes(T, 4000, 256), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.gemm_w8a8(a, sa, w, sw, out=out, ws=ws)
        ops.gemm_w8a8(a, sa, w, sw, out=out, ws=ws)
    a.copy_(torch.flip(a, [0]))
    sa.copy_(torch.flip(sa, [0]))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, torch.flip(want, [0]))


@gpu
def test_nan_scales_and_no_rows():
    """A token whose scale is NaN (a row the norm could not scale) gives a row of NaN, and no other."""
    from bit_moe_expert_route_gb300 import ops
    for T in (4, 90):
        a, sa, w, sw = inputs(T, 200, 64, 1)
        sa[2] = float("nan")
        nan = torch.isnan(ops.gemm_w8a8(a, sa, w, sw))
        assert nan[2].all() and nan.sum() == 200
        assert ops.gemm_w8a8(a[:0], sa[:0], w, sw).shape == (0, 200)


@pytest.fixture(scope="module")
def L():
    from bit_moe_expert_route_gb300 import build as B
    B.build()
    from bit_moe_expert_route_gb300 import ops
    return ops.lib()


def test_refusals(L):
    buf = np.zeros(1 << 16, np.uint8)
    p = (buf.ctypes.data + 255) // 256 * 256
    vp = ctypes.c_void_p

    def call(a=p, lda=64, sa=p, w=p, sw=p, T=2, N=8, K=64, type=0, out=p, ldo=8, ws=p, n=4096):
        return L.moe_gemm_w8a8(vp(a), lda, vp(sa), vp(w), vp(sw), T, N, K, type, vp(out), ldo, vp(ws), n, None)
    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(K=72, lda=80), dict(K=65552, lda=65552), dict(lda=48), dict(lda=72), dict(ldo=7),
                dict(type=2), dict(type=-1)):
        assert call(**bad) == -3, bad
    for bad in ("a", "sa", "w", "sw", "out"):
        assert call(**{bad: None}) == -1, bad
    for bad in (dict(a=p + 8), dict(w=p + 4), dict(sa=p + 2), dict(sw=p + 1), dict(out=p + 1), dict(out=p + 2, type=1)):
        assert call(**bad) == -2, bad
    for bad in (dict(ws=None, T=100, N=20000, ldo=20000), dict(ws=p + 16), dict(n=255), dict(T=100, N=20000, ldo=20000, n=256)):
        assert call(**bad) == -4, bad
    assert call(T=0, a=None) == 0
    assert L.moe_gemm_w8a8_workspace_bytes(100, 20000, 64) >= 256 + 100 * 64 * 2
    assert L.moe_gemm_w8a8_workspace_bytes(24, 1 << 20, 64) == 256
    assert L.moe_gemm_w8a8_workspace_bytes(1, 8, 60) == 0


def test_binding_refuses_wrong_tensors():
    from bit_moe_expert_route_gb300 import ops
    a, s = torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError, match="int8"):
        ops.gemm_w8a8(a.float(), s, a, s)
    with pytest.raises(ValueError, match="GPU"):
        ops.gemm_w8a8(a, s, a, s)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        ops.gemm_w8a8(a, s, a, s, dtype=torch.float16)

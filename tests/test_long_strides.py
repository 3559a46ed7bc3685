"""The operators around the layer on rows whose offsets pass 32 bits: strided views of one
buffer of 2.9e9 elements. Values against the same call on compact copies, bit for bit (the
rows' distance changes no order of sums)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
LD = 4_200_000  # elements from row to row
ROWS = 700


@pytest.fixture(scope="module")
def pool():
    p = torch.empty(ROWS * LD, dtype=torch.bfloat16, device="cuda")
    yield p
    del p
    torch.cuda.empty_cache()


def rows(pool, dtype, n, width, seed, offset=0):
    """n rows of `width` elements of `dtype`, as far apart as the buffer lets them be."""
    flat = pool.view(dtype)
    ld = flat.numel() // ROWS
    v = flat.as_strided((n, width), (ld, 1), offset)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype is torch.int8:
        v.copy_(torch.randint(-127, 128, (n, width), generator=g, device="cuda").to(dtype))
    else:
        v.copy_(torch.randn(n, width, generator=g, device="cuda").to(dtype))
    return v


def test_norm(pool):
    from bit_moe_expert_route_gb300 import ops
    x = rows(pool, torch.bfloat16, ROWS, 264, 1)
    w = torch.ones(264, device="cuda").bfloat16()
    a, b = ops.add_rmsnorm_q8(x, w), ops.add_rmsnorm_q8(x.contiguous(), w)
    assert torch.equal(a.q, b.q) and torch.equal(a.scale, b.scale)


@pytest.mark.parametrize("T,N", [(20, 300), (ROWS, 300), (ROWS, 20000)])
def test_product(pool, T, N):
    """Rows of tokens and of the output both far apart."""
    from bit_moe_expert_route_gb300 import ops
    a = rows(pool, torch.int8, T, 256, 2)
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randint(-127, 128, (N, 256), generator=g, device="cuda").to(torch.int8)
    sa, sw = torch.rand(T, device="cuda"), torch.rand(N, device="cuda")
    want = ops.gemm_w8a8(a.contiguous(), sa, w, sw)
    out = pool.as_strided((T, N), (LD, 1), 1000)
    ops.gemm_w8a8(a, sa, w, sw, out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [300, 40000])
def test_logprobs(pool, dtype, V):
    from bit_moe_expert_route_gb300 import ops
    z = rows(pool, dtype, ROWS, V, 3, offset=1)
    ids = torch.arange(ROWS, dtype=torch.int32, device="cuda") % V
    a, b = ops.token_logprobs(z, ids, top_k=7), ops.token_logprobs(z.contiguous(), ids, top_k=7)
    assert torch.equal(a.top_ids, b.top_ids)
    # the rows' alignment, and with it the order of the sums, differs: within both calls' 2e-5
    assert torch.all((a.logprob - b.logprob).abs() <= 4e-5) and torch.all((a.entropy - b.entropy).abs() <= 2e-4)


@pytest.mark.parametrize("B,P,S", [(2, 600, 40), (2, ROWS, 0), (40, ROWS, 0), (30, 300, 20), (3, 0, 200)])
def test_attention(pool, B, P, S):
    """Positions far apart (the sequences' own: position s of sequence b in row b S + s)."""
    from bit_moe_expert_route_gb300 import ops
    q = torch.randn(B, 8, 64, device="cuda").bfloat16()
    kp = rows(pool, torch.bfloat16, max(P, 1), 128, 4)[:P].unflatten(1, (2, 64))
    vp = rows(pool, torch.bfloat16, max(P, 1), 128, 5, offset=1024)[:P].unflatten(1, (2, 64))
    n = min(S, ROWS // B)
    ks = rows(pool, torch.bfloat16, B * n, 128, 6, offset=2048).view(B, n, 2, 64) if n else None
    vs = rows(pool, torch.bfloat16, B * n, 128, 7, offset=4096).view(B, n, 2, 64) if n else None
    ln = torch.randint(0, n + 1, (B,), dtype=torch.int32, device="cuda") if n else None
    got = ops.prefix_attention(q, kp, vp, ks, vs, ln)
    want = ops.prefix_attention(q, kp.contiguous(), vp.contiguous(), ks.contiguous() if n else None, vs.contiguous() if n else None, ln)
    assert torch.equal(got, want) and got.abs().sum() > 0

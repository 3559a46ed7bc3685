"""moe_qk_norm_rope against its formula in 64 bits.

A pair's output is a cos - b sin or a sin + b cos of its normed elements a, b. In fp32: the
mean of up to 256 squares, a root, a quotient and two products, 2^-20 of each element at most;
cos and sin to 2^-22, a product and a fused sum, below 2^-21 of |a| + |b| more. The store's rounding is half a step of
bf16, 2^-8 of the value at most. Per element |err| <= 2^-8 |o| + 2^-19 (|a| + |b|).
"""
import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


def axis_of(pairs, sections, cyclic):
    A = len(sections)
    if cyclic:
        return [i % A if i < A * sections[i % A] else 0 for i in range(pairs)]
    return [a for a, n in enumerate(sections) for _ in range(n)]


def expected(x, weight, eps, rope=None, positions=None):
    """(o, |a| + |b|) in 64 bits; x [T, H, d]."""
    y = x.double()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    o, mag = y.clone(), y.abs()
    if rope is not None:
        n = rope.freqs.numel()
        sections = rope.sections or (n,)
        at = positions.view(len(sections), -1)[axis_of(n, sections, rope.cyclic)].t().double()
        ang = (at * rope.freqs.double())[:, None]
        ia = torch.arange(n, device=x.device) * (2 if rope.adjacent else 1)
        ib = ia + (1 if rope.adjacent else n)
        a, b = y[..., ia], y[..., ib]
        o[..., ia], o[..., ib] = a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return o, mag


def check(got, o, mag):
    assert torch.all((got.double() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -19 * mag + 1e-38)


def inputs(T, Hq, Hkv, d, seed, wide=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device="cuda").mul(1.5).bfloat16()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    w = [torch.randn(d, generator=g, device="cuda").mul(0.3).add(1).bfloat16() for _ in range(2)]
    return (q, k) if wide else (q.contiguous(), k.contiguous()), w, g


SHAPES = [  # T, Hq, Hkv, d, pairs, sections, cyclic, adjacent, norm, far
    (1, 16, 2, 256, 32, None, False, False, True, 40000), (1, 1, 1, 8, 4, None, False, True, True, 10),
    (3, 3, 1, 24, 8, None, False, False, True, 1000), (5, 7, 1, 16, 8, None, False, False, False, 1 << 20),
    (700, 32, 8, 128, 64, (16, 24, 24), False, False, True, 5000), (65, 32, 8, 128, 64, (24, 20, 20), True, False, True, 5000),
    (130, 8, 8, 64, 32, (32,), False, False, False, 1 << 30), (33, 12, 4, 128, 64, (10, 30, 20, 4), False, True, True, 1 << 30),
    (33, 12, 4, 128, 64, (40, 8, 8, 8), True, True, True, 100000), (257, 5, 3, 80, 16, None, False, False, True, 100000),
    (19, 9, 1, 96, 48, (48, 0), False, False, True, 3000), (4000, 16, 2, 256, 128, None, False, False, True, 1 << 31),
    (77, 2, 2, 120, 60, None, False, True, False, 7), (9, 16, 2, 256, 32, (0, 32), False, False, True, 999), (2500, 1, 1, 64, 16, (6, 5, 5), True, False, True, 50)]


@gpu
@pytest.mark.parametrize("T,Hq,Hkv,d,pairs,sections,cyclic,adjacent,norm,far", SHAPES)
def test_matches_64_bits(T, Hq, Hkv, d, pairs, sections, cyclic, adjacent, norm, far):
    from bit_moe_expert_route_gb300 import ops
    (q, k), (wq, wk), g = inputs(T, Hq, Hkv, d, T + d)
    rope = ops.Rope(ops.rope_freqs(2 * pairs, 1e6), sections, cyclic, adjacent)
    A = len(sections or (0,))
    at = torch.randint(-far, far, (A, T), generator=g, device="cuda").clamp(max=2 ** 31 - 1).to(torch.int32)
    at[:, 0] = 0
    at[:, -1] = far - 1
    if not norm:
        wq = wk = None
    gq, gk = ops.qk_norm_rope(q, k, rope, at if A > 1 else at[0], wq, wk, eps=1e-5)
    check(gq, *expected(q, wq, 1e-5, rope, at))
    check(gk, *expected(k, wk, 1e-5, rope, at))


@gpu
@pytest.mark.parametrize("d", [8, 64, 72, 256])
def test_parts_alone(d):
    """Queries alone, norm alone, a weight for one of the two, neither; and no tokens."""
    from bit_moe_expert_route_gb300 import ops
    (q, k), (wq, wk), g = inputs(37, 6, 2, d, d)
    gq, gk = ops.qk_norm_rope(q, k, None, None, wq)
    check(gq, *expected(q, wq, 1e-6))
    assert torch.equal(gk, k)
    gq, none = ops.qk_norm_rope(q, q_weight=wq)
    assert none is None
    check(gq, *expected(q, wq, 1e-6))
    assert torch.equal(ops.qk_norm_rope(q)[0], q)
    a, b = ops.qk_norm_rope(q[:0], k[:0], None, None, wq, wk)
    assert a.shape == (0, 6, d) and b.shape == (0, 2, d)


@gpu
def test_one_position_for_all_axes():
    """Positions of three axes that are one row of memory (text among patches), or a slice of a wider tensor."""
    from bit_moe_expert_route_gb300 import ops
    (q, k), (wq, wk), g = inputs(50, 8, 2, 128, 4)
    rope, at = ops.Rope(ops.rope_freqs(128), (16, 24, 24)), torch.arange(50, dtype=torch.int32, device="cuda")
    a = ops.qk_norm_rope(q, k, rope, at.expand(3, 50), wq, wk)
    wide = torch.zeros(3, 70, dtype=torch.int32, device="cuda")
    wide[:, 5:55] = at
    b = ops.qk_norm_rope(q, k, rope, wide[:, 5:55], wq, wk)
    c = ops.qk_norm_rope(q, k, ops.Rope(rope.freqs), at, wq, wk)
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))


@gpu
def test_in_place_and_into_views():
    from bit_moe_expert_route_gb300 import ops
    (q, k), (wq, wk), g = inputs(300, 16, 2, 128, 1)
    rope, at = ops.Rope(ops.rope_freqs(64)), torch.arange(300, dtype=torch.int32, device="cuda")
    want = ops.qk_norm_rope(q, k, rope, at, wq, wk)
    out = torch.full((300, 25, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.qk_norm_rope(q, k, rope, at, wq, wk, q_out=out[:, 1:17], k_out=out[:, 20:22])
    assert torch.equal(out[:, 1:17], want[0]) and torch.equal(out[:, 20:22], want[1])
    assert torch.all(out[:, [0, 17, 18, 19, 22, 23, 24]] == 7)
    base = q.as_strided((300, 20, 128), (20 * 128, 128, 1)).clone()
    views = base[:, :16], base[:, 16:18]
    got = ops.qk_norm_rope(*views, rope, at, wq, wk, q_out=views[0], k_out=views[1])
    assert torch.equal(got[0], want[0]) and torch.equal(base[:, :16], want[0]) and torch.equal(base[:, 16:18], want[1])
    assert torch.equal(base[:, 18:], q.as_strided((300, 20, 128), (20 * 128, 128, 1))[:, 18:])


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_extreme_rows(d):
    """Zeros; rows whose squares pass fp32 or vanish in it; a NaN or an infinity in one head."""
    from bit_moe_expert_route_gb300 import ops
    (q, k), (wq, wk), g = inputs(12, 4, 2, d, 5, wide=False)
    q[1] = 0
    q[2] *= 1e37
    q[3] *= 1e-30
    q[4, 0] *= 2e19
    q[5, :, ::2] *= 1e38 / 6
    rope, at = ops.Rope(ops.rope_freqs(d)), torch.arange(12, dtype=torch.int32, device="cuda") * 1000
    got = ops.qk_norm_rope(q, None, rope, at, wq)[0]
    o, mag = expected(q, wq, 1e-6, rope, at)
    check(got, o, mag)
    assert not got[1].any() and torch.isfinite(got).all()
    q[6, 2, 5], q[7, 3, 0] = float("nan"), float("inf")
    odd = torch.zeros(12, 4, dtype=torch.bool, device="cuda")
    odd[6, 2] = odd[7, 3] = True
    bad = ops.qk_norm_rope(q, None, rope, at, wq)[0]
    assert torch.equal(bad[~odd], got[~odd]) and torch.isnan(bad[6, 2]).all()
    assert torch.isnan(bad[7, 3, [0, d // 2]]).all() and not bad[7, 3, 1:d // 2].any()
    freqs = rope.freqs.clone()
    freqs[3] = float("nan")
    bad = ops.qk_norm_rope(q[:6], None, ops.Rope(freqs), at[:6], wq)[0]
    assert torch.isnan(bad[..., [3, 3 + d // 2]]).all() and torch.isfinite(bad[..., 4:d // 2]).all()


@gpu
def test_long_strides():
    """Tokens whose offsets pass 2^31 elements."""
    from bit_moe_expert_route_gb300 import ops
    (q, k), (wq, wk), g = inputs(3, 2, 1, 64, 3)
    rope, at = ops.Rope(ops.rope_freqs(64)), torch.arange(3, dtype=torch.int32, device="cuda")
    ld = (1 << 30) + 64
    far = torch.empty(2 * ld + 2 * 64, dtype=torch.bfloat16, device="cuda").as_strided((3, 2, 64), (ld, 64, 1))
    far.copy_(q)
    want = ops.qk_norm_rope(q, k, rope, at, wq, wk)[0]
    assert torch.equal(ops.qk_norm_rope(far, None, rope, at, wq)[0], want)
    ops.qk_norm_rope(far, None, rope, at, wq, q_out=far)
    assert torch.equal(far, want)
    del far
    torch.cuda.empty_cache()


@gpu
def test_graph_and_stream():
    """Captured and replayed with other inputs; on another stream."""
    from bit_moe_expert_route_gb300 import ops
    (q, k), (wq, wk), g = inputs(50, 16, 2, 256, 9)
    rope, at = ops.Rope(ops.rope_freqs(64)), torch.arange(50, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.qk_norm_rope(q, k, rope, at, wq, wk, q_out=outs[0], k_out=outs[1])
    for step in (1, 77):
        at += step
        q.mul_(0.5)
        graph.replay()
        want = ops.qk_norm_rope(q, k, rope, at, wq, wk)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        other = ops.qk_norm_rope(q, k, rope, at, wq, wk, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(outs, want, other))

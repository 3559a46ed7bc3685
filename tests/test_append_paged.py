"""moe_append_paged: keys within the rounding of test_qk_norm_rope, values and everything that is not
written bit for bit."""
import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16)


def after(P, k, v, rows=None, weight=None, rope=None, positions=None, left_out=()):
    """(K pool in 64 bits, its |a| + |b|, V pool, where something was written)."""
    from test_qk_norm_rope import expected
    kp, vp = P.cache.k_pages.double(), P.cache.v_pages.clone()
    mag, done = torch.zeros_like(kp), torch.zeros(kp.shape[:2], dtype=torch.bool, device="cuda")
    for b, (a, n) in enumerate(zip(P.lens_list, P.news)):
        for i in range(n):
            t = P.starts_list[b] + i
            if t in left_out:
                continue
            r = t if rows is None else int(rows[t])
            page, place = (int(x) for x in P.places(b, [a + i]))
            at = torch.tensor([[a + i]], device="cuda") if positions is None else positions.view(-1, P.N)[:, t:t + 1]
            o, m = expected(k[r:r + 1], weight, 1e-6, rope, at)
            kp[page, place], mag[page, place], vp[page, place], done[page, place] = o[0], m[0], v[r], True
    return kp, mag, vp, done


def check(P, want, before):
    from test_qk_norm_rope import check as near
    kp, mag, vp, done = want
    near(P.cache.k_pages[done], kp[done], mag[done])
    assert torch.equal(bits(P.cache.v_pages), bits(vp))
    assert torch.equal(bits(P.cache.k_pages[~done]), bits(before[~done]))


CASES = [  # lens, news, Hkv, d, page, order, pairs, adjacent, norm
    ([4000], [1], 2, 256, 16, "places", 32, False, True), ([0], [1], 1, 8, 8, "places", 4, True, False),
    ([0, 5, 0, 31, 32, 100], [3, 0, 40, 1, 33, 0], 8, 128, 32, "places", 64, False, True),
    ([0, 5, 0, 31, 32, 100], [3, 0, 40, 1, 33, 0], 8, 128, 32, "heads", 64, False, True),
    ([7, 0, 90], [5, 70, 1], 2, 64, 64, "pair", 0, False, False), ([7, 0, 90], [5, 70, 1], 3, 64, 8, "heads", 16, True, True),
    ([300, 0], [0, 200], 1, 256, 4096, "places", 128, False, False), ([5000], [130], 4, 80, 128, "pair", 16, False, True),
    (list(range(40)), [b % 3 for b in range(40)], 2, 128, 16, "places", 64, False, True)]


@gpu
@pytest.mark.parametrize("lens,news,Hkv,d,page,order,pairs,adjacent,norm", CASES)
def test_places_and_values(lens, news, Hkv, d, page, order, pairs, adjacent, norm):
    from bit_moe_expert_route_gb300 import ops
    from paged import Paged
    P = Paged(lens, news, Hkv, d, page, 3, order, stale=5.0)
    qkv = P.normal(P.N, 2 * Hkv + 3, d, std=1.5)
    k, v = qkv[:, 1:1 + Hkv], qkv[:, 2 + Hkv:2 + 2 * Hkv]
    rope = ops.Rope(ops.rope_freqs(2 * pairs, 1e5), adjacent=adjacent) if pairs else None
    w = P.normal(d, std=0.2) + 1 if norm else None
    before = P.cache.k_pages.clone()
    want = after(P, k, v, weight=w, rope=rope)
    ops.append_paged(k, v, P.cache, P.starts, P.lens, rope, k_weight=w)
    check(P, want, before)


@gpu
def test_rows_and_positions():
    """Paths of trees appended again: rows out of order, twice, and outside; tokens' own positions of
    three axes."""
    from bit_moe_expert_route_gb300 import ops
    from paged import Paged
    P = Paged([10, 3, 77], [4, 1, 9], 2, 128, 16, 5, stale=1.0)
    k, v = P.normal(30, 2, 128), P.normal(30, 2, 128)
    rows = torch.tensor([29, 0, 3, 3, -1, 7, 8, 30, 9, 1 << 30, 28, 11, 12, -(1 << 31)], dtype=torch.int32, device="cuda")
    rope = ops.Rope(ops.rope_freqs(128), (16, 24, 24))
    at = torch.randint(0, 5000, (3, P.N), generator=P.g, device="cuda", dtype=torch.int32)
    before = P.cache.k_pages.clone()
    want = after(P, k, v, rows, None, rope, at, left_out=(4, 7, 9, 13))
    ops.append_paged(k, v, P.cache, P.starts, P.lens, rope, at, rows=rows)
    check(P, want, before)


@gpu
def test_what_has_no_place_is_left_out():
    """Tokens before the first start and behind the last, pages outside the pool, positions past the
    table, negative lengths."""
    from bit_moe_expert_route_gb300 import ops
    from paged import Paged
    P = Paged([10, 20, 0, 40], [30, 30, 8, 8], 2, 64, 16, 6, stale=2.0)
    n = P.cache.k_pages.shape[0]
    k, v = P.normal(P.N, 2, 64), P.normal(P.N, 2, 64)
    left = set(range(0, 4)) | set(range(70, 76))
    P.starts[0], P.starts[4] = 4, 70           # tokens 0-3 and 70-75 are nobody's
    P.lens_list[0], P.lens[0] = 10, 10
    P.starts_list[0] = 4
    P.news[0], P.news[3] = 26, 2
    P.table[1, 2], P.cache.table[1, 2] = n, n     # positions 32-47 of sequence 1
    left |= {30 + i for i in range(30) if 32 <= 20 + i < 48}
    P.lens[2] = -9                              # counts as 0
    P.cache.table[3, 2] = -1                    # positions 32-47 of sequence 3
    left |= {68, 69}
    before = P.cache.k_pages.clone()
    fixed = P.table.clone()
    P.table[1, 2] = 0
    want = after(P, k, v, left_out=left)
    P.table = fixed
    ops.append_paged(k, v, P.cache, P.starts, P.lens)
    check(P, want, before)
    # past the table: nothing is written
    P.lens.fill_(2 ** 31 - 40)
    held = bits(P.cache.k_pages).clone()
    ops.append_paged(k, v, P.cache, P.starts, P.lens)
    assert torch.equal(bits(P.cache.k_pages), held)
    ops.append_paged(k[:0], v[:0], P.cache, torch.zeros_like(P.starts), P.lens)
    assert torch.equal(bits(P.cache.k_pages), held)


@gpu
@pytest.mark.parametrize("B", [31, 32, 33, 1000, 1025, 40000])
def test_many_sequences(B):
    """The search for a token's sequence, empty ones among them."""
    from bit_moe_expert_route_gb300 import ops
    d, page = 8, 8
    host = torch.Generator().manual_seed(B)
    news = torch.randint(0, 3, (B,), generator=host)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), news.cumsum(0)])
    N = int(starts[-1])
    k = torch.arange(N * d, device="cuda").remainder(251).view(N, 1, d).bfloat16()
    pages = torch.zeros(B, page, 1, d, dtype=torch.bfloat16, device="cuda")
    cache = ops.PagedCache(pages, torch.zeros_like(pages), torch.arange(B, dtype=torch.int32, device="cuda")[:, None])
    ops.append_paged(k, -k, cache, starts.int().cuda(), torch.full((B,), 3, dtype=torch.int32, device="cuda"))
    want = torch.zeros_like(pages)
    for i in range(2):
        has = (news > i).cuda()
        want[has, 3 + i] = k[(starts[:-1].cuda() + i)[has]]
    assert torch.equal(pages, want) and torch.equal(cache.v_pages, -want)


@gpu
def test_far_pages():
    """Pages whose offsets pass 2^31 elements."""
    from bit_moe_expert_route_gb300 import ops
    page, d, n = 8, 64, 5
    ps = (1 << 30) + 64
    buf = torch.empty((n - 1) * ps + 2 * page * d, dtype=torch.bfloat16, device="cuda")
    kp, vp = (buf[o:].as_strided((n, page, 1, d), (ps, d, d, 1)) for o in (0, page * d))
    kp.zero_(), vp.zero_()
    cache = ops.PagedCache(kp, vp, torch.tensor([[4, 1]], dtype=torch.int32, device="cuda"))
    k = torch.randn(12, 1, d, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    ops.append_paged(k, -k, cache, torch.tensor([0, 12], **i32), torch.tensor([0], **i32))
    assert torch.equal(kp[4], k[:8]) and torch.equal(kp[1, :4], k[8:]) and torch.equal(vp[4], -k[:8]) and torch.equal(vp[1, :4], -k[8:])
    assert not kp[0].any() and not kp[2:4].any() and not kp[1, 4:].any()
    del buf, kp, vp, cache
    torch.cuda.empty_cache()


@gpu
def test_graph_and_stream():
    from bit_moe_expert_route_gb300 import ops
    from paged import Paged
    P = Paged([10, 3, 77], [4, 1, 9], 2, 128, 16, 5, stale=1.0, extra=1)
    k, v = P.normal(P.N, 2, 128), P.normal(P.N, 2, 128)
    rope, w = ops.Rope(ops.rope_freqs(128)), P.normal(128)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.append_paged(k, v, P.cache, P.starts, P.lens, rope, k_weight=w)
    for step in range(2):
        k.mul_(-0.5)
        P.lens_list = [n - 3 * step for n in P.lens_list]
        P.lens.sub_(3 * step)
        before, want = P.cache.k_pages.clone(), after(P, k, v, weight=w, rope=rope)
        graph.replay()
        check(P, want, before)
        copies = [t.clone() for t in P.cache[:2]]
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        ops.append_paged(k, v, P.cache, P.starts, P.lens, rope, k_weight=w, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(copies, P.cache[:2]))

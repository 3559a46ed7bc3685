"""moe_tree_attention against softmax attention in 64 bits.

The fp32 scores of up to 256 products leave each weight within 1e-3 for these inputs (256 *
2^-24 of a sum of magnitudes below 60), the weights' two bf16 parts within 2^-16 of it, and the output
is rounded to bf16 (2^-8 of it at most): per element |err| <= 2^-8 |o| + 1.1e-3 sum_j p_j |v_j|. Over a
whole output the roundings are independent, uniform within 2^-8 of a value at most: 2^-8 / sqrt(3) =
2.26e-3 of the 2-norm, and 3e-4 for the rest.
"""
import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


def seen(P, tree, b):
    """[n, L + n]: what each new token of a sequence attends to."""
    L, n, t0 = P.lens_list[b], P.news[b], P.starts_list[b]
    m = torch.ones(n, L + n, dtype=torch.bool)
    for i in range(n):
        for j in range(n):
            m[i, L + j] = j <= i if tree is None else bool(int(tree[t0 + i]) >> j & 1)
    return m.cuda()


def expected(P, q, tree, scale=None):
    """(o, sum_j p_j |v_j|) in 64 bits; rows that attend to nothing are zeros."""
    N, Hq, d = q.shape
    G = Hq // P.Hkv
    scale = scale or d ** -0.5
    o = torch.zeros(N, Hq, d, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(o)
    tree = None if tree is None else tree.cpu()
    for b, n in enumerate(P.news):
        if not n:
            continue
        t0, m = P.starts_list[b], seen(P, tree, b).repeat_interleave(G, dim=0)
        k, v = (t.double() for t in P.read(b))
        some = m.any(dim=1)
        for h in range(P.Hkv):
            rows = q[t0:t0 + n, h * G:(h + 1) * G].reshape(n * G, d).double()
            # positions out of sight play no part, whatever they hold
            s = torch.where(m, rows @ k[:, h].t() * scale, torch.tensor(float("-inf"), dtype=torch.float64, device="cuda"))
            p = torch.where(some[:, None], torch.softmax(s, dim=1), torch.zeros_like(s))
            used = torch.where(m.any(dim=0)[:, None], v[:, h], torch.zeros_like(v[:, h]))
            o[t0:t0 + n, h * G:(h + 1) * G] = (p @ used).view(n, G, d)
            mag[t0:t0 + n, h * G:(h + 1) * G] = (p @ used.abs()).view(n, G, d)
    return o, mag


def check(got, o, mag):
    err = (got.double() - o).abs()
    assert torch.all(err <= 2.0 ** -8 * o.abs() + 1.1e-3 * mag), float((err / mag.clamp(min=1e-30)).max())
    assert float(err.norm()) <= 2.56e-3 * float(o.norm())


def paged(lens, news, Hq, Hkv, d, page, seed=0, tree=True, order="places", **more):
    from paged import Paged, random_tree
    P = Paged(lens, news, Hkv, d, page, seed, order, **more).fill()
    return P, P.normal(P.N, Hq, d, std=1.5), random_tree(news, seed) if tree else None


def call(P, q, tree, **more):
    """The output, from a workspace of 0xFF, with its status checked."""
    from bit_moe_expert_route_gb300 import ops
    args = ops._paged_args("test", P.cache, P.Hkv, P.d, 0)[0]
    ws = torch.full((ops.lib().moe_tree_attention_workspace_bytes(q.shape[0], q.shape[1], args),), 255,
                    dtype=torch.uint8, device="cuda")
    out = ops.tree_attention(q, P.cache, P.starts, P.lens, tree, ws=ws, **more)
    assert ops.device_status(ws) == 0
    return out


CASES = [  # lens, news, Hq, Hkv, d, page, tree
    ([0], [1], 1, 1, 64, 8, False), ([1], [1], 16, 2, 256, 16, False), ([700], [5], 16, 2, 256, 16, True),
    ([0], [64], 16, 1, 128, 64, True), ([63], [1], 4, 4, 128, 32, False), ([64, 127, 128], [1, 1, 1], 8, 8, 64, 128, False),
    ([65, 0, 4000, 129, 300], [3, 0, 64, 1, 17], 12, 4, 128, 16, True), ([5, 70, 0, 0, 190], [64, 63, 2, 0, 0], 16, 1, 64, 8, True),
    ([100, 2000, 30, 77], [20, 9, 64, 2], 6, 2, 256, 32, True), ([100, 2000, 30, 77], [20, 9, 64, 2], 32, 2, 256, 64, True),
    ([3000], [64], 16, 1, 256, 256, False), ([30011], [3], 16, 2, 128, 512, True), ([9001, 20, 3], [8, 8, 8], 32, 8, 128, 4096, True),
    ([7 * b % 100 for b in range(200)], [b % 4 for b in range(200)], 8, 2, 64, 16, True),
    ([b % 3 for b in range(700)], [1 + b % 2 for b in range(700)], 4, 4, 64, 8, False), ([60000], [16], 16, 2, 256, 64, True),
    ([1000 + 37 * b for b in range(64)], [1] * 64, 32, 8, 128, 64, False), ([1000 + 37 * b for b in range(40)], [13] * 40, 8, 8, 64, 32, True),
    ([8000 - 300 * b for b in range(8)], [16] * 8, 16, 2, 256, 128, True)]


@gpu
@pytest.mark.parametrize("lens,news,Hq,Hkv,d,page,tree", CASES, ids=lambda x: str(x)[:30])
def test_matches_64_bits(lens, news, Hq, Hkv, d, page, tree):
    from bit_moe_expert_route_gb300 import ops
    P, q, tree = paged(lens, news, Hq, Hkv, d, page, sum(lens) + d, tree)
    got = call(P, q, tree)
    check(got, *expected(P, q, tree))
    assert torch.equal(ops.tree_attention(q, P.cache, P.starts, P.lens, tree), got)  # the merge order is fixed


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("order", ["heads", "pair"])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_layouts_and_scale(d, order, page):
    """Positions inside heads; K and V side by side; queries out of a wider buffer."""
    P, q, tree = paged([300, 40, 1000], [7, 1, 30], 15, 3, d, page, d, True, order)
    wide = torch.zeros(P.N, 17, d, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:16] = q
    check(call(P, wide[:, 1:16], tree, scale=0.2), *expected(P, q, tree, 0.2))


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("L", [0, 1, 63, 64, 100, 127, 128, 191, 3000])
def test_what_is_out_of_sight_plays_no_part(d, L):
    """New tokens that no row, or not every row, attends to hold NaN and infinities in K and V; rows
    that attend to them show it, the others do not. Masks without bits; bits past the last token."""
    P, q, tree = paged([L, L + 1], [64, 9], 4, 2, d, 16, L + d)
    host = torch.Generator().manual_seed(L)
    bits = [[int(torch.randint(0, 2, (1,), generator=host)) for _ in range(64)] for _ in range(73)]
    words = []
    for t, w in enumerate(bits):
        w[3] = w[40] = 0                 # tokens that nobody attends to
        m = 0 if t in (5, 66) else sum(x << j for j, x in enumerate(w))
        if t >= 64:
            m |= 0x55 << 40              # (that sequence has 9 tokens)
        words.append(m - (1 << 64) if m >> 63 else m)
    tree = torch.tensor(words, dtype=torch.int64, device="cuda")
    clean = tree.clone()
    clean[64:] &= 511
    want = expected(P, q, clean)
    kp, vp = P.cache.k_pages, P.cache.v_pages
    (p3, o3), (p40, o40) = (tuple(int(x) for x in P.places(0, [L + j])) for j in (3, 40))
    kp[p3, o3], vp[p3, o3] = float("nan"), float("inf")
    kp[p40, o40, 1], vp[p40, o40, 0, ::3] = float("inf"), float("nan")
    got = call(P, q, tree)
    check(got, *want)
    if L == 0:
        assert not got[5].any()
    # one that some attend to: its V shows in their rows alone, in its own columns
    to = tuple(int(x) for x in P.places(0, [L + 20]))
    vp[to][0, 1], vp[to][1, 6], vp[to][1, 7] = float("inf"), float("nan"), float("-inf")
    see = torch.tensor([w[20] == 1 and t != 5 for t, w in enumerate(bits)], device="cuda")
    see[64:] = False
    bad = call(P, q, tree)
    hit = torch.zeros_like(got, dtype=torch.bool)
    for h, c in ((0, 1), (1, 6), (1, 7)):
        hit[see, 2 * h:2 * h + 2, c] = True
    assert torch.equal(bad[~hit], got[~hit])
    assert torch.all(bad[see][:, :2, 1] == float("inf")) and torch.all(bad[see][:, 2:, 7] == float("-inf"))
    assert torch.isnan(bad[see][:, 2:, 6]).all() and see.any() and not see.all()


@gpu
@pytest.mark.parametrize("d", [64, 256])
def test_infinite_and_nan_scores(d):
    P, q, tree = paged([500, 20], [6, 40], 8, 2, d, 16, d)
    q[1, 5, 3] = float("nan")
    got = call(P, q, tree)
    bad = torch.zeros(P.N, 8, dtype=torch.bool, device="cuda")
    bad[1, 5] = True
    assert torch.isnan(got[bad]).all() and torch.isfinite(got[~bad]).all()
    q[1, 5, 3] = 1.0
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    to = tuple(int(x) for x in P.places(0, [77]))
    P.cache.k_pages[to][0, 0] = float("-inf")  # every score of this key is -infinity
    check(call(P, q, tree), *expected(P, q, tree))
    P.cache.k_pages[to][0, 0] = float("inf")
    got = call(P, q, tree)
    assert torch.isnan(got[:6, :4]).all() and torch.isfinite(got[:6, 4:]).all() and torch.isfinite(got[6:]).all()
    to = P.places(1, range(60))
    P.cache.k_pages[to[0], to[1], :, 0] = float("-inf")
    got = call(P, q, tree)
    assert not got[6:].any()


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lowest_and_large_scores(d):
    """Keys of the type's lowest and largest values, far ahead of the rest and behind it."""
    P, q, tree = paged([300, 70], [5, 9], 4, 2, d, 32, d)
    q.zero_()
    q[..., 0] = 1.0
    lowest = torch.finfo(torch.bfloat16).min
    for b, at in ((0, range(0, 290)), (1, range(0, 60))):
        to = P.places(b, at)
        P.cache.k_pages[to[0], to[1], :, 0] = lowest
    check(call(P, q, tree), *expected(P, q, tree))
    to = P.places(0, [3])
    P.cache.k_pages[to[0], to[1], :, 0] = 1e30
    check(call(P, q, tree), *expected(P, q, tree))


@gpu
def test_tokens_of_no_sequence():
    """Rows before the first start and behind the last are left as they were."""
    P, q, tree = paged([100, 300], [4, 6], 8, 2, 128, 16, 3)
    wide = torch.randn(25, 8, 128, device="cuda").bfloat16()
    wide[7:17] = q
    masks = torch.full((25,), -1, dtype=torch.int64, device="cuda")
    masks[7:17] = tree
    starts = P.starts
    want = call(P, q, tree)
    P.starts = starts + 7
    out = torch.full_like(wide, 7.0)
    call(P, wide, masks, out=out)
    assert torch.equal(out[7:17], want) and torch.all(out[:7] == 7) and torch.all(out[17:] == 7)
    P.starts = torch.zeros_like(starts)
    out.fill_(7.0)
    call(P, wide, masks, out=out)
    assert torch.all(out == 7)
    from bit_moe_expert_route_gb300 import ops
    assert ops.tree_attention(q[:0], P.cache, P.starts, P.lens, tree[:0]).shape == (0, 8, 128)


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_sequences_that_cannot_be_right(d):
    """A page outside the pool, positions past the table, more than 64 new tokens: NaN for that
    sequence alone. Negative lengths count as 0."""
    P, q, tree = paged([900, 200, 400, 30], [4, 6, 70, 2], 8, 2, d, 16, 3, tree=False)
    P.news[2] = 64
    want = expected(P, q, None)  # (of the third, not all: not looked at)
    n = P.cache.k_pages.shape[0]
    got = call(P, q, None)
    s = P.starts_list
    assert torch.isnan(got[s[2]:s[3]]).all()
    for bad in (n, -1, 2 ** 31 - 1, -2 ** 31):
        held = int(P.cache.table[0, 30])
        P.cache.table[0, 30] = bad
        got = call(P, q, None)
        P.cache.table[0, 30] = held
        assert torch.isnan(got[:s[1]]).all()
        for b in (1, 3):
            check(got[s[b]:s[b + 1]], *(t[s[b]:s[b + 1]] for t in want))
    for far in (P.cache.table.shape[1] * 16 - 5, 2 ** 31 - 1):
        P.lens[1] = far
        got = call(P, q, None)
        assert torch.isnan(got[s[1]:s[2]]).all()
        for b in (0, 3):
            check(got[s[b]:s[b + 1]], *(t[s[b]:s[b + 1]] for t in want))
    P.lens[1], P.lens_list[1] = -5, 0
    got, want = call(P, q, None), expected(P, q, None)
    check(got[s[1]:s[2]], *(t[s[1]:s[2]] for t in want))


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_graph_whose_lengths_change(d):
    """Captured once; replayed after the caches grew, with other masks and other counts of new tokens."""
    P, q, tree = paged([300, 40, 1000], [7, 1, 30], 8, 2, d, 32, d, extra=2)
    out = torch.empty_like(q)
    call(P, q, tree)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    from bit_moe_expert_route_gb300 import ops
    with torch.cuda.graph(graph):
        ops.tree_attention(q, P.cache, P.starts, P.lens, tree, out=out)
    graph.replay()
    torch.cuda.synchronize()
    check(out, *expected(P, q, tree))
    from paged import random_tree
    P.lens_list, P.news = [280, 45, 90], [20, 0, 18]
    P.starts_list = [0, 20, 20, 38]
    P.lens.copy_(torch.tensor(P.lens_list)), P.starts.copy_(torch.tensor(P.starts_list))
    tree.copy_(random_tree(P.news, 4))
    q.mul_(0.7)
    graph.replay()
    torch.cuda.synchronize()
    check(out, *expected(P, q, tree))


@gpu
def test_two_streams_at_once():
    """Two calls with workspaces of their own run side by side."""
    from bit_moe_expert_route_gb300 import ops
    A = paged([5000] * 4, [9] * 4, 16, 2, 128, 64, 1)
    B = paged([200, 9000], [3, 64], 16, 2, 256, 16, 2)
    want = [call(P, q, t) for P, q, t in (A, B)]
    s, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (P, q, t) in enumerate((A, B)):
            got[i].append(ops.tree_attention(q, P.cache, P.starts, P.lens, t, stream=s[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])


@gpu
def test_far_pages():
    """Pages and queries whose offsets pass 2^31 elements."""
    from bit_moe_expert_route_gb300 import ops
    P, q, tree = paged([70], [5], 8, 2, 128, 16, 1, spare=0)
    n = P.cache.k_pages.shape[0]
    ps = (1 << 30) // 128 * 128
    buf = torch.empty((n - 1) * ps + 2 * 16 * 256, dtype=torch.bfloat16, device="cuda")
    kp, vp = (buf[o:].as_strided((n, 16, 2, 128), (ps, 256, 128, 1)) for o in (0, 16 * 256))
    kp.copy_(P.cache.k_pages), vp.copy_(P.cache.v_pages)
    ld = (1 << 29) + 8
    far = torch.empty(4 * ld + 1024, dtype=torch.bfloat16, device="cuda").as_strided((5, 8, 128), (ld, 128, 1))
    far.copy_(q)
    assert 4 * ld >= 1 << 31 and (n - 1) * ps >= 1 << 31
    want = call(P, q, tree)
    got = ops.tree_attention(far, ops.PagedCache(kp, vp, P.cache.table), P.starts, P.lens, tree)
    assert torch.equal(got, want)
    del buf, kp, vp, far
    torch.cuda.empty_cache()


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_shared_pages_and_one_pool(d):
    """Sequences whose first pages are the same ones; a pool that is keys and values both."""
    P, q, tree = paged([400, 170, 333], [5, 64, 1], 8, 2, d, 32, 9)
    P.table[1:, :5] = P.table[0, :5]
    P.cache.table.copy_(P.table)
    check(call(P, q, tree), *expected(P, q, tree))
    P.cache = P.cache._replace(v_pages=P.cache.k_pages)
    check(call(P, q, tree), *expected(P, q, tree))

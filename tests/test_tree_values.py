"""moe_tree_attention where values are infinite or NaN: whose rows show it, and as what."""
import pytest

torch = pytest.importorskip("torch")
from test_tree_attention import call, check, expected, paged  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
def test_segment_after_segment_of_odd_values(d):
    """Many short sequences, each of whose new tokens has an infinite value of its own: a block goes from one such
    sequence to the next, and every row shows its own infinities, in every warp's rows."""
    news = [64, 1, 9, 33] * 40
    P, q, tree = paged([b % 7 for b in range(160)], news, 4, 2, d, 16, d, tree=False)
    finite = call(P, q, None)
    hit = torch.zeros_like(finite, dtype=torch.bool)
    for b, n in enumerate(news):
        at = (3 * b) % n
        to = tuple(int(x) for x in P.places(b, [P.lens_list[b] + at]))
        P.cache.v_pages[to][b % 2, (5 * b) % d] = float("inf")
        hit[P.starts_list[b] + at:P.starts_list[b] + n, 2 * (b % 2):2 * (b % 2) + 2, (5 * b) % d] = True
    for _ in range(5):
        got = call(P, q, None)
        assert torch.all(got[hit] == float("inf")) and torch.equal(got[~hit], finite[~hit])


def odd_expected(P, q, tree):
    """(o, sum_j p_j |v_j|) in 64 bits of finite values, and what infinities and NaN that rows attend to add."""
    from test_tree_attention import seen
    held = P.cache.v_pages.clone()
    P.cache.v_pages.masked_fill_(~torch.isfinite(held), 0.0)
    o, mag = expected(P, q, tree)
    P.cache.v_pages.copy_(held)
    odd = torch.zeros_like(o)
    G = q.shape[1] // P.Hkv
    for b, n in enumerate(P.news):
        if n:
            v = P.read(b)[1].double()
            places = (~torch.isfinite(v)).any(dim=2).any(dim=1).nonzero()[:, 0]
            add = torch.where(torch.isfinite(v[places]), 0.0, v[places])  # [odd, Hkv, d]
            m = seen(P, tree, b)[:, places]
            rows = torch.where(m[:, :, None, None], add[None], 0.0).sum(dim=1)
            odd[P.starts_list[b]:P.starts_list[b] + n] = rows.repeat_interleave(G, dim=1)
    return o, mag, odd


def check_odd(got, o, mag, odd):
    assert torch.equal(torch.isnan(got), torch.isnan(odd))
    inf = torch.isinf(odd)
    assert inf.any() and torch.equal(got[inf].double(), odd[inf])
    finite = odd == 0
    check(got[finite], o[finite], mag[finite])


CACHED = [  # lens, news, Hq, Hkv, page, tree: short (whole in one block), in parts, more than one row tile
    ([1], [1], 1, 1, 8, False), ([70], [5], 16, 2, 16, True), ([300, 129, 64], [1, 64, 7], 8, 2, 32, True),
    ([40000], [1], 16, 2, 64, False), ([30011, 5], [40, 3], 16, 2, 128, True), ([257 + b for b in range(50)], [1] * 50, 32, 8, 16, False)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,news,Hq,Hkv,page,tree", CACHED, ids=lambda x: str(x)[:20])
def test_infinite_values_of_cached_positions(lens, news, Hq, Hkv, page, tree, d):
    """An infinity of a cached value shows as that infinity in its column of every row, not as the NaN that a
    weight's second part, negative or 0, would make of it; both signs or a NaN as NaN; with those of new tokens."""
    P, q, tree = paged(lens, news, Hq, Hkv, d, page, sum(lens) + d, tree)
    inf, host = float("inf"), torch.Generator().manual_seed(d)

    def put(b, position, head, column, value):
        to = tuple(int(x) for x in P.places(b, [position]))
        P.cache.v_pages[to][head, column] = value
    for b, (L, n) in enumerate(zip(lens, news)):
        at = [int(torch.randint(0, L, (1,), generator=host)) for _ in range(6)]
        put(b, 0, 0, 0, inf), put(b, L - 1, Hkv - 1, d - 1, -inf), put(b, at[0], 0, 5, inf), put(b, at[1], Hkv - 1, 17, -inf)
        put(b, at[2], 0, 33, inf), put(b, (at[2] + 1) % L, 0, 34, -inf)
        if L > 1:
            put(b, at[3], 0, 40, inf), put(b, (at[3] + 1) % L, 0, 40, -inf)
            put(b, at[4], Hkv - 1, 41, float("nan"))
        # with new tokens' (the last one, which some rows attend to): the same sign, the other, one alone
        put(b, L + n - 1, 0, 5, inf), put(b, L + n - 1, 0, 33, -inf), put(b, L + n - 1, 0, 50, -inf)
    got = call(P, q, tree)
    check_odd(got, *odd_expected(P, q, tree))
    assert torch.equal(call(P, q, tree).view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("below", ["far", "infinitely"])
@pytest.mark.parametrize("L", [90, 30000])
def test_infinite_values_of_positions_without_weight(L, below, d):
    """Positions whose weights are 0 in fp32, or exactly (scores of -infinity), in a block of their own or in one with the
    largest score: what is infinite there shows all the same. A row of nothing but -infinity is zeros."""
    P, q, tree = paged([L, 40], [5, 9], 8, 2, d, 16, d)
    q[..., 0] = 1.0
    for b, last in ((0, L), (1, 40)):
        to = P.places(b, range(last))
        P.cache.k_pages[to[0], to[1], :, 0] = 0.0
    if below == "far":
        to = P.places(0, range(10))
        P.cache.k_pages[to[0], to[1], :, 0] = 300.0 * d ** 0.5   # 300 above the rest: e^-300
    else:
        to = P.places(0, range(10, L + 5))
        P.cache.k_pages[to[0], to[1], :, 0] = float("-inf")
    for at, column in ((L - 7, 3), (L // 2 + 20, 4), (L, 5), (L + 4, 6)):
        to = tuple(int(x) for x in P.places(0, [at]))
        P.cache.v_pages[to][:, column] = float("inf")
    got = call(P, q, tree)
    check_odd(got, *odd_expected(P, q, tree))
    to = P.places(0, range(L + 5))
    P.cache.k_pages[to[0], to[1], :, 0] = float("-inf")
    assert not call(P, q, tree)[:5].any()

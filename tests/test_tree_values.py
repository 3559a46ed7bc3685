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

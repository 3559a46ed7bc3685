"""Sizes that 32 bits do not hold, or whose products they would not: refused, not wrapped."""
import pytest

torch = pytest.importorskip("torch")
from test_cache_arguments import SHAPE, L, append, norm, rope  # noqa: E402, F401


@pytest.mark.parametrize("pairs", [1 << 30, (1 << 30) + 8, (1 << 31) - 8])
def test_pairs_whose_double_wraps(L, pairs):  # noqa: F811
    """2^30 pairs would be -2^31 elements, fewer than a head has."""
    import fake_cuda as F
    for axes, sections in ((1, None), (2, (pairs - 8, 8)), (4, (pairs, 0, 0, 0))):
        for adjacent in (0, 1):
            r = rope(pairs=pairs, axes=axes, sections=sections, adjacent=adjacent)
            assert norm(L, r=r) == SHAPE and append(L, r=r) == SHAPE
    assert F.launches(L) == []

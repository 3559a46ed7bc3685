"""Pools whose strides are not multiples of one another, or whose pages lie inside positions: appended to and
attended to as a pool in plain order is, bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PADDED = {  # strides of (page, place, head) in elements, from (pages, page, heads, d)
    "positions with a rest": lambda n, page, H, d: ((H * d + 8) * page, H * d + 8, d),
    "pages with a rest": lambda n, page, H, d: (page * H * d + 24, H * d, d),
    "heads with a rest": lambda n, page, H, d: (((d + 40) * H + 16) * page + 8, (d + 40) * H + 16, d + 40),
    "positions inside heads, rests": lambda n, page, H, d: (H * (page * (d + 8) + 8) + 56, d + 8, page * (d + 8) + 8),
    "pages inside positions": lambda n, page, H, d: (H * d, n * H * d, d),
    "pages inside positions, rests": lambda n, page, H, d: (H * d + 8, n * (H * d + 8) + 72, d),
    "pages inside heads": lambda n, page, H, d: (page * d, d, n * page * d),
}


def strided(t, strides, fill):
    """A copy of t [n, page, H, d] at strides of its first three axes, and the memory around it."""
    n = 1 + sum((size - 1) * s for size, s in zip(t.shape, strides + (1,)))
    memory = torch.full((n,), fill, dtype=t.dtype, device=t.device)
    view = memory.as_strided(t.shape, strides + (1,))
    view.copy_(t)
    return view, memory


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("layout", PADDED)
def test_strides(layout, H, d):
    from bit_moe_expert_route_gb300 import ops
    from test_tree_attention import call, paged
    P, q, tree = paged([300, 40, 129], [7, 1, 30], 2 * H, H, d, 16, d)
    plain = P.cache
    k, v, w = P.normal(P.N, H, d), P.normal(P.N, H, d), P.normal(d)
    rope = ops.Rope(ops.rope_freqs(d))
    strides = PADDED[layout](*plain.k_pages.shape)
    (kp, kmem), (vp, vmem) = (strided(t, strides, 3.0) for t in plain[:2])
    other = ops.PagedCache(kp, vp, plain.table)
    whole = torch.zeros_like(kmem, dtype=torch.bool)
    whole.as_strided(kp.shape, kp.stride()).fill_(True)
    for cache in (plain, other):
        ops.append_paged(k, v, cache, P.starts, P.lens, rope, k_weight=w)
    for a, b, memory in ((plain.k_pages, kp, kmem), (plain.v_pages, vp, vmem)):
        assert torch.equal(a.view(torch.int16), b.contiguous().view(torch.int16)) and torch.all(memory[~whole] == 3.0)
    want = call(P, q, tree)
    P.cache = other
    assert torch.equal(call(P, q, tree), want)

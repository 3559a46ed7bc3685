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


class Tensor:
    """A tensor on cuda:0 of which only the description exists."""
    device, is_cuda = "cuda:0", True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, torch.Size(shape)
        steps = [1]
        for n in reversed(shape[1:]):
            steps.insert(0, steps[0] * n)
        self.steps = tuple(steps)

    def get_device(self):
        return 0

    def stride(self, i=None):
        return self.steps if i is None else self.steps[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def test_sizes_that_the_call_would_wrap(monkeypatch):
    """2^32 + 5 tokens of one small head fit the card; as 32 bits they are 5."""
    from bit_moe_expert_route_gb300 import ops
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)

    class Library:
        def __getattr__(self, name):
            def called(*args):
                raise AssertionError(f"{name} is called")
            return called
    monkeypatch.setattr(ops, "_lib", Library())
    bf, i32, far = torch.bfloat16, torch.int32, (1 << 32) + 5

    def refused(fn, *args, **more):
        with pytest.raises(ValueError, match="too large"):
            fn(*args, **more)
    for n in (1 << 31, far):
        q = Tensor(bf, n, 1, 8)
        refused(ops.qk_norm_rope, q, q_out=q)
        q = Tensor(bf, 1, n, 8)
        refused(ops.qk_norm_rope, q, q_out=q)
        q = Tensor(bf, 1, 1, n)
        refused(ops.qk_norm_rope, q, q_out=q)
        q, k = Tensor(bf, 3, 1, 8), Tensor(bf, 3, n, 8)
        refused(ops.qk_norm_rope, q, k, q_out=q, k_out=k)
        pages = Tensor(bf, 4, 16, 1, 8)
        cache = ops.PagedCache(pages, pages, Tensor(i32, 1, 4))
        k = Tensor(bf, n, 1, 8)
        refused(ops.append_paged, k, k, cache, Tensor(i32, 2), Tensor(i32, 1))
        refused(ops.append_paged, k, k, cache, Tensor(i32, 2), Tensor(i32, 1), rows=Tensor(i32, 7))
        k = Tensor(bf, 7, 1, 8)
        refused(ops.append_paged, k, k, cache, Tensor(i32, 2), Tensor(i32, 1), rows=Tensor(i32, n))
        q = Tensor(bf, n, 1, 8)
        refused(ops.tree_attention, q, cache, Tensor(i32, 2), Tensor(i32, 1), out=q, ws=Tensor(torch.uint8, 1 << 20))
        q = Tensor(bf, 3, 1, 8)
        r = ops.Rope(Tensor(torch.float32, n))
        refused(ops.qk_norm_rope, q, None, r, Tensor(i32, 3), q_out=q)

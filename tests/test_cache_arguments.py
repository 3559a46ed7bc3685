"""What the paged cache's operators refuse, without a GPU: through the C ABI (addresses that nothing
reads: a call that passes its checks goes to a runtime that launches nothing) and through the binding."""
import ctypes
import shutil

import pytest

torch = pytest.importorskip("torch")
A = 1 << 20  # an address
SHAPE, NULL, ALIGN, WS = -3, -1, -2, -4


@pytest.fixture(scope="module")
def L():
    if not shutil.which("g++"):
        pytest.skip("the fake runtime needs g++")
    import fake_cuda as F
    from bit_moe_expert_route_gb300 import ops
    lib, real = F.lib(), ops.lib()
    for name in ("moe_qk_norm_rope", "moe_append_paged", "moe_tree_attention_workspace_bytes", "moe_tree_attention"):
        f, g = getattr(lib, name), getattr(real, name)
        f.argtypes, f.restype = g.argtypes, g.restype
    return lib


def rope(freqs=A, positions=A, ld=1 << 20, pairs=32, axes=1, sections=None, cyclic=0, adjacent=0):
    from bit_moe_expert_route_gb300 import ops
    s = list(sections or (pairs,))
    return ops._ROPE_ARGS.pack(freqs or 0, positions or 0, ld, pairs, axes, *(s + [0] * 4)[:4], cyclic, adjacent)


def cache(k=A, v=A, ps=16 * 2 * 128, os=2 * 128, hs=128, table=A, ld=10, n=50, page=16, width=10, B=3, H=2, d=128):
    from bit_moe_expert_route_gb300 import ops
    return ops._PAGED_ARGS.pack(k or 0, v or 0, ps, os, hs, table or 0, ld, n, page, width, B, H, d)


def norm(L, q=A, ldq=2048, k=A, ldk=256, T=10, Hq=16, Hkv=2, d=128, wq=A, wk=A, eps=1e-6, r="one", qo=A, ldqo=2048, ko=A, ldko=256):
    return L.moe_qk_norm_rope(q, ldq, k, ldk, T, Hq, Hkv, d, wq, wk, eps, rope() if r == "one" else r, qo, ldqo, ko, ldko, None)


def test_norm_and_rotation(L):
    assert norm(L) == 0 and norm(L, T=0, q=None, k=None, qo=None, ko=None) == 0
    assert norm(L, r=None, wq=None, wk=None) == 0
    assert norm(L, k=None, ldk=0, Hkv=0, ko=None, ldko=0, wk=None) == 0
    assert norm(L, q=None, ldq=0, Hq=0, qo=None, ldqo=0) == 0
    for bad in (dict(T=-1), dict(Hq=-1), dict(d=4), dict(d=100), dict(d=264, ldq=1 << 20, ldk=1 << 20), dict(ldq=2040), dict(ldq=2052),
                dict(ldk=248), dict(ldqo=2040), dict(ldko=12), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(T=(1 << 31) // 18 + 1), dict(ldq=1 << 39)):
        assert norm(L, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None)):
        assert norm(L, **bad) == NULL, bad
    for bad in (dict(q=A + 8), dict(k=A + 2), dict(qo=A + 8), dict(ko=A + 8), dict(wq=A + 2), dict(wk=A + 8)):
        assert norm(L, **bad) == ALIGN, bad
    for bad in (dict(pairs=-8), dict(pairs=68), dict(pairs=72), dict(pairs=20), dict(pairs=10, adjacent=1), dict(axes=0), dict(axes=5),
                dict(axes=3, sections=(10, 10, 10)), dict(axes=2, sections=(-8, 40)), dict(axes=2, sections=(40, -8)),
                dict(axes=3, sections=(8, 12, 12), cyclic=1), dict(axes=3, sections=(16, 8, 8), ld=-1),
                dict(axes=2, sections=((1 << 31) - 1, 33))):
        assert norm(L, r=rope(**bad)) == SHAPE, bad
    for good in (dict(pairs=0), dict(pairs=64), dict(pairs=12, adjacent=1), dict(axes=3, sections=(12, 10, 10), cyclic=1),
                 dict(axes=4, sections=(0, 0, 32, 0)), dict(axes=3, sections=(16, 8, 8), ld=0)):
        assert norm(L, r=rope(**good)) == 0, good
    assert norm(L, r=rope(freqs=None)) == NULL and norm(L, r=rope(positions=None)) == NULL
    assert norm(L, r=rope(freqs=A + 2)) == ALIGN and norm(L, r=rope(positions=A + 1)) == ALIGN


def append(L, k=A, ldk=256, v=A, ldv=256, rows=None, n_rows=10, N=10, starts=A, lens=A, c=None, w=A, eps=1e-6, r="one"):
    return L.moe_append_paged(k, ldk, v, ldv, rows, n_rows, N, starts, lens, cache() if c is None else c, w, eps,
                              rope() if r == "one" else r, None)


BAD_CACHES = [dict(n=0), dict(n=-1), dict(page=4), dict(page=24), dict(page=8192), dict(page=0), dict(width=0), dict(width=-3),
              dict(B=0), dict(B=65536), dict(H=0), dict(H=1025, ps=1 << 20, os=1 << 18), dict(ps=120), dict(ps=4100), dict(os=4), dict(hs=12), dict(hs=0),
              dict(os=1 << 39), dict(ps=-4096), dict(ld=9), dict(width=1 << 25, ld=1 << 25)]


def test_appending(L):
    assert append(L) == 0 and append(L, r=None, w=None) == 0 and append(L, rows=A, n_rows=3) == 0
    assert append(L, N=0, n_rows=0, k=None, v=None, starts=None, lens=None) == 0
    assert append(L, rows=A, n_rows=0, k=None, v=None) == 0  # (every row is outside)
    assert append(L, r=rope(positions=None)) == 0
    for bad in (dict(N=-1, n_rows=-1), dict(n_rows=9), dict(n_rows=11), dict(rows=A, n_rows=-1), dict(ldk=248), dict(ldv=260),
                dict(eps=0.0), dict(N=1 << 30, n_rows=1 << 30)):
        assert append(L, **bad) == SHAPE, bad
    assert append(L, r=rope(positions=None, axes=3, sections=(16, 8, 8))) == SHAPE
    for bad in BAD_CACHES:
        assert append(L, c=cache(**bad)) == SHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(starts=None), dict(lens=None)):
        assert append(L, **bad) == NULL, bad
    for bad in (dict(k=None), dict(v=None), dict(table=None)):
        assert append(L, c=cache(**bad)) == NULL, bad
    for bad in (dict(k=A + 8), dict(v=A + 8), dict(rows=A + 2), dict(starts=A + 1), dict(lens=A + 2), dict(w=A + 8)):
        assert append(L, **bad) == ALIGN, bad
    for bad in (dict(k=A + 8), dict(v=A + 2), dict(table=A + 2)):
        assert append(L, c=cache(**bad)) == ALIGN, bad
    assert L.moe_append_paged(A, 256, A, 256, None, 10, 10, A, A, None, A, 1e-6, None, None) == NULL
    # strides of axes of one entry say nothing
    assert append(L, c=cache(H=1, hs=3, os=128, ps=2048)) == 0 and append(L, c=cache(n=1, ps=5)) == 0 and append(L, c=cache(B=1, ld=1)) == 0


def tree(L, q=A, ldq=2048, N=10, Hq=16, starts=A, lens=A, bits=A, c=None, scale=0.0, out=A, ws=A, n=None):
    c = cache() if c is None else c
    if n is None:
        n = L.moe_tree_attention_workspace_bytes(N, Hq, c)
    return L.moe_tree_attention(q, ldq, N, Hq, starts, lens, bits, c, scale, out, ws, n, None)


def test_attention(L):
    import fake_cuda as F
    for d in (64, 128, 256):
        L.fake_reset()
        c = dict(d=d, hs=d, os=2 * d, ps=32 * d)
        assert tree(L, c=cache(**c), ldq=16 * d) == 0
        (k, grid, *_), (m, merge, *_) = F.launches(L)
        assert k == f"tree_kernel<{d}>" and m == f"tree_merge_kernel<{d}>" and grid[0] == 152 and merge[0] == 608
        need = L.moe_tree_attention_workspace_bytes(10, 16, cache(**c))
        assert need >= 2 * 152 * 80 * (d + 2) * 4 and tree(L, c=cache(**c), ldq=16 * d, n=need - 1) == WS
        for order in (dict(os=d, hs=16 * d, ps=32 * d), dict(os=4 * d, hs=d, ps=64 * d)):
            assert tree(L, c=cache(**dict(c, **order)), ldq=16 * d) == 0
    assert tree(L, N=0, q=None, out=None, starts=None, lens=None, ws=None) == 0 and tree(L, bits=None) == 0
    for bad in (dict(N=-1), dict(N=1 << 24), dict(Hq=15), dict(Hq=1), dict(Hq=34, ldq=1 << 14), dict(ldq=2040), dict(ldq=2052),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38)):
        assert tree(L, **bad, n=1 << 30) == SHAPE, bad
    for bad in BAD_CACHES + [dict(d=96, hs=96, os=192, ps=16 * 192)]:
        assert tree(L, c=cache(**bad), n=1 << 30) == SHAPE and L.moe_tree_attention_workspace_bytes(10, 16, cache(**bad)) == 0, bad
    for bad in (dict(q=None), dict(out=None), dict(starts=None), dict(lens=None)):
        assert tree(L, **bad) == NULL, bad
    for bad in (dict(q=A + 8), dict(out=A + 2), dict(starts=A + 2), dict(lens=A + 1), dict(bits=A + 4)):
        assert tree(L, **bad) == ALIGN, bad
    assert tree(L, ws=None) == WS and tree(L, ws=A + 16) == WS
    # the largest sizes
    assert tree(L, N=(1 << 24) - 1, c=cache(B=65535, width=1 << 21, page=128, ld=1 << 21, ps=1 << 20)) == 0
    assert append(L, N=(1 << 29) - 1, n_rows=(1 << 29) - 1) == 0 and norm(L, T=(1 << 31) // 18 - 1) == 0


def test_every_device_and_a_failed_opt_in(L):
    for d in (64, 128, 256):
        c = dict(d=d, hs=d, os=2 * d, ps=32 * d)
        for dev in (1, 0, 5, 90):
            L.fake_set_device(dev)
            assert tree(L, c=cache(**c), ldq=16 * d) == 0
        for dev in (40, 100):
            L.fake_set_device(dev)
            L.fake_fail_attributes(1)
            assert tree(L, c=cache(**c), ldq=16 * d) != 0
            assert tree(L, c=cache(**c), ldq=16 * d) == 0
    L.fake_set_device(0)


def test_masks_of_a_tree():
    from bit_moe_expert_route_gb300 import ops
    bits, depths = ops.tree_masks([-1, 0, 0, 1, -1, 3])
    assert bits.tolist() == [1, 3, 5, 11, 16, 43] and depths.tolist() == [0, 1, 1, 2, 0, 3]
    assert bits.dtype == torch.int64 and depths.dtype == torch.int32
    chain, depths = ops.tree_masks(range(-1, 63))
    assert chain[63] == -1 and chain[62] == (1 << 63) - 1 and depths[63] == 63
    assert ops.tree_masks([])[0].shape == (0,)
    for bad in ([0], [-2], [-1, 1], [-1] * 65):
        with pytest.raises(ValueError, match="tree_masks"):
            ops.tree_masks(bad)


def test_frequencies():
    from bit_moe_expert_route_gb300 import ops
    f = ops.rope_freqs(8, 1e4, device="cpu")
    assert f.dtype == torch.float32 and torch.equal(f, torch.tensor([1.0, 0.1, 0.01, 0.001]))


def test_the_binding_refuses_what_is_not_on_the_gpu():
    from bit_moe_expert_route_gb300 import ops
    bf = torch.bfloat16
    q, pages = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(5, 16, 2, 64, dtype=bf)
    c = ops.PagedCache(pages, pages, torch.zeros(1, 2, dtype=torch.int32))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="qk_norm_rope: q .* on the GPU"):
        ops.qk_norm_rope(q)
    with pytest.raises(ValueError, match="rope without positions"):
        ops.qk_norm_rope(q, rope=ops.Rope(torch.ones(8)))
    with pytest.raises(ValueError, match="without k"):
        ops.qk_norm_rope(q, k_weight=torch.ones(64, dtype=bf))
    with pytest.raises(ValueError, match="append_paged: k .* on the GPU"):
        ops.append_paged(q[:, :2], q[:, :2], c, i, i[:1])
    with pytest.raises(ValueError, match="tree_attention: q .* on the GPU"):
        ops.tree_attention(q, c, i, i[:1])


@pytest.mark.gpu
def test_the_binding_refuses():
    from bit_moe_expert_route_gb300 import ops
    bf, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    q, k = torch.zeros(3, 4, 64, **bf), torch.zeros(3, 2, 64, **bf)
    pages, at = torch.zeros(5, 16, 2, 64, **bf), torch.zeros(3, **i32)
    table, starts, lens = torch.zeros(1, 2, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    c, r = ops.PagedCache(pages, pages.clone(), table), ops.Rope(ops.rope_freqs(64))

    def refused(match, fn, *args, **more):
        with pytest.raises(ValueError, match=match):
            fn(*args, **more)
    n, a, t = ops.qk_norm_rope, ops.append_paged, ops.tree_attention
    refused("q is", n, q.float())
    refused("q has scattered", n, q.transpose(1, 2).contiguous().transpose(1, 2))
    refused("q has scattered", n, torch.zeros(3, 8, 64, **bf)[:, ::2])
    refused("k is", n, q, k[:2])
    refused("q_weight", n, q, q_weight=torch.ones(63, **bf))
    refused("k_weight", n, q, k, k_weight=torch.ones(64, device="cuda"))
    refused("q_out", n, q, q_out=q[:, :3])
    refused("positions", n, q, k, r, at[:2])
    refused("positions", n, q, k, r, at.long())
    refused("positions", n, q, k, ops.Rope(r.freqs, (16, 8, 8)), at)
    refused("positions without rope", n, q, k, None, at)
    refused("rope.freqs", n, q, k, ops.Rope(r.freqs.double()), at)
    refused("rope.freqs", n, q, k, ops.Rope(r.freqs.cpu()), at)
    refused("5 sections", n, q, k, ops.Rope(r.freqs, (8, 8, 8, 8, 0)), at)
    with pytest.raises(ops.MoeError):
        n(q, k, ops.Rope(ops.rope_freqs(128)), at)
    refused("v is", a, k, k[:, :1], c, starts, lens)
    refused("k_pages is", a, k[:, :1], k[:, :1], c, starts, lens)
    refused("k_pages", a, k, k, ops.PagedCache(pages[0], pages[0], table), starts, lens)
    refused("v_pages is", a, k, k, ops.PagedCache(pages, pages[:4], table), starts, lens)
    refused("different strides", a, k, k, ops.PagedCache(pages, torch.zeros(5, 2, 16, 64, **bf).transpose(1, 2), table), starts, lens)
    refused("table", a, k, k, ops.PagedCache(pages, pages, table.long()), starts, lens)
    refused("table", a, k, k, ops.PagedCache(pages, pages, table[0]), starts, lens)
    refused("starts", a, k, k, c, starts[:1], lens)
    refused("lens", a, k, k, c, starts, starts)
    refused("rows", a, k, k, c, starts, lens, rows=at.long())
    refused("q is", t, q.half(), c, starts, lens)
    refused("k_pages is", t, torch.zeros(3, 4, 128, **bf), c, starts, lens)
    refused("tree", t, q, c, starts, lens, at)
    refused("out", t, q, c, starts, lens, out=q.float())
    refused("ws", t, q, c, starts, lens, ws=torch.zeros(1 << 24, dtype=torch.uint8))
    with pytest.raises(ops.MoeError):
        t(q, c, starts, lens, ws=torch.zeros(1 << 10, dtype=torch.uint8, device="cuda"))
    odd = torch.zeros(8 * 16 * 24 * 64, **bf)[4:4 + 5 * 16 * 2 * 64].view(5, 16, 2, 64)
    with pytest.raises(ops.MoeError):
        t(q, ops.PagedCache(odd, odd, table), starts, lens)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """What is on another device than the call's other tensors, or than the current one, whose stream the
    call would go to."""
    from bit_moe_expert_route_gb300 import ops

    class Elsewhere:
        device, dtype, shape, is_cuda = "cuda:1", torch.int32, (3,), True

        def get_device(self):
            return 1

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 64
    assert ops._vector("f", "x", Elsewhere(), torch.int32, 3, 1) == 64
    with pytest.raises(ValueError, match="f: x is on cuda:1, the call's other tensors on cuda:0"):
        ops._vector("f", "x", Elsewhere(), torch.int32, 3, 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 7, raising=False)
    assert ops._current("f", 0) == 7
    with pytest.raises(ValueError, match="f: the tensors are on cuda:1, cuda:0 is the current device"):
        ops._current("f", 1)


def test_the_structures_are_the_headers():
    """What the binding packs lies as a C compiler lays the header's structures out."""
    import os
    import subprocess
    import tempfile
    from bit_moe_expert_route_gb300 import ops
    from bit_moe_expert_route_gb300 import build as B
    src = r"""#include <stdio.h>
#include <stddef.h>
#include "cache.h"
int main() {
  printf("%zu %zu %zu %zu %zu\n", sizeof(moe_rope_t), offsetof(moe_rope_t, ld_positions), offsetof(moe_rope_t, pairs), offsetof(moe_rope_t, sections), offsetof(moe_rope_t, adjacent));
  printf("%zu %zu %zu %zu\n", sizeof(moe_paged_t), offsetof(moe_paged_t, page_stride), offsetof(moe_paged_t, table), offsetof(moe_paged_t, n_pages));
}
"""
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "s.c"), os.path.join(d, "s")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", B.INCLUDE, c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [ops._ROPE_ARGS.size, 16, 24, 32, 52, ops._PAGED_ARGS.size, 16, 40, 56]

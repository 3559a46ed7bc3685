"""moe_prefix_attention against softmax attention in 64 bits.

The softmax weights are rounded to bf16 (half a step, 2^-8 of each) before they
multiply the values, the output is rounded to bf16 (2^-8 of it), and the fp32
scores of up to 256 products leave each weight within 1e-3 for these inputs
(256 * 2^-24 of a sum of magnitudes below 60): per element
|err| <= 2^-8 |o| + (2^-8 + 1e-3) sum_j p_j |v_j|. Over a whole output the
roundings are independent, with rms 0.41 * 2^-8 each: 4e-3 in the 2-norm
holds with room.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


def inputs(B, P, S, Hq, Hkv, d, seed, lens=None):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul(std).bfloat16()
    if lens is None:
        lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    else:
        lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return n(B, Hq, d, std=1.5), n(P, Hkv, d), n(P, Hkv, d), n(B, S, Hkv, d), n(B, S, Hkv, d), lens


def expected(q, kp, vp, ks, vs, lens, scale=None):
    B, Hq, d = q.shape
    Hkv = kp.shape[1]
    G = Hq // Hkv
    scale = scale or d ** -0.5
    o, mag = torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device), torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(lens[b].clamp(0, ks.shape[1])) if ks is not None else 0
        for h in range(Hkv):
            k, v = kp[:, h].double(), vp[:, h].double()
            if n:
                k, v = torch.cat([k, ks[b, :n, h].double()]), torch.cat([v, vs[b, :n, h].double()])
            if len(k):
                p = torch.softmax(q[b, h * G:(h + 1) * G].double() @ k.t() * scale, dim=1)
                o[b, h * G:(h + 1) * G], mag[b, h * G:(h + 1) * G] = p @ v, p @ v.abs()
    return o, mag


def check(got, o, mag):
    err = (got.double() - o).abs()
    assert torch.all(err <= 2.0 ** -8 * o.abs() + (2.0 ** -8 + 1e-3) * mag), float((err / mag.clamp(min=1e-30)).max())
    assert float(err.norm()) <= 4e-3 * float(o.norm())


SHAPES = [(1, 1, 1, 2, 2, 64), (1, 0, 5, 16, 2, 256), (3, 64, 0, 16, 2, 128), (2, 700, 16, 16, 2, 256), (1, 65, 1, 4, 4, 64),
          (5, 129, 33, 12, 4, 128), (8, 8192, 200, 32, 8, 128), (9, 1000, 70, 16, 1, 64), (17, 333, 130, 8, 8, 64), (64, 2049, 65, 16, 2, 256),
          (33, 500, 9, 6, 2, 256), (2, 30000, 3, 3, 1, 128), (1, 20000, 3000, 16, 2, 256), (40, 0, 300, 8, 1, 128), (150, 90, 20, 16, 2, 64),
          (4, 4096, 64, 16, 1, 256),
          # more than 32 rows a KV head and at least 256 shared positions: the tensor-memory kernel
          (70, 512, 0, 3, 3, 64), (16, 513, 3, 16, 2, 128), (40, 1000, 30, 8, 2, 128), (13, 700, 10, 16, 1, 256), (20, 4099, 10, 12, 2, 256),
          (65, 9000, 70, 2, 2, 128), (100, 30011, 9, 10, 1, 64), (64, 20000, 100, 16, 2, 256), (5, 256, 40, 16, 2, 128), (33, 257, 0, 2, 2, 64), (5, 700, 70, 16, 2, 256),
          # little work: one launch of clusters of 1 to 8 blocks, the prefix ending inside a tile or at its end
          (1, 0, 1, 16, 1, 256), (7, 10, 50, 4, 4, 128), (4, 100, 28, 16, 1, 64), (3, 128, 64, 6, 2, 128), (2, 1900, 100, 16, 2, 64),
          (9, 515, 1, 12, 4, 128), (19, 1983, 65, 2, 2, 256), (1, 2048, 0, 8, 8, 64)]


@gpu
@pytest.mark.parametrize("B,P,S,Hq,Hkv,d", SHAPES)
def test_matches_64_bits(B, P, S, Hq, Hkv, d):
    from bit_moe_expert_route_gb300 import ops
    x = inputs(B, P, S, Hq, Hkv, d, B + P + S + d)
    ws = torch.empty(ops.lib().moe_prefix_attention_workspace_bytes(B, P, S, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    got = ops.prefix_attention(*x, ws=ws)
    assert ops.device_status(ws) == 0
    check(got, *expected(*x))
    assert torch.equal(ops.prefix_attention(*x), got)  # the merge order is fixed


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_stale_positions_are_not_read(d):
    """Positions past a sequence's length hold NaN and infinities; lengths are clamped to 0 .. S."""
    from bit_moe_expert_route_gb300 import ops
    lens = [0, 1, 63, 64, 65, 130, -3, 4000]
    q, kp, vp, ks, vs, ln = inputs(8, 70, 130, 8, 2, d, d, lens)
    for b, n in enumerate(lens):
        n = min(max(n, 0), 130)
        ks[b, n:], vs[b, n:] = float("nan"), float("inf")
    check(ops.prefix_attention(q, kp, vp, ks, vs, ln), *expected(q, kp, vp, ks, vs, ln))


@gpu
def test_rows_without_positions_are_zero():
    from bit_moe_expert_route_gb300 import ops
    q, kp, vp, ks, vs, ln = inputs(4, 0, 40, 16, 2, 128, 1, [0, 7, 0, 40])
    got = ops.prefix_attention(q, kp, vp, ks, vs, ln)
    assert not got[0].any() and not got[2].any()
    check(got, *expected(q, kp, vp, ks, vs, ln))
    assert not ops.prefix_attention(q, kp, vp).any()  # neither a prefix nor suffixes
    assert ops.prefix_attention(q[:0], kp, vp, ks[:0], vs[:0], ln[:0]).shape == (0, 16, 128)


@gpu
@pytest.mark.parametrize("B,d", [(3, 64), (3, 256), (30, 64), (30, 128), (30, 256)])
def test_bad_queries_and_infinite_keys(B, d):
    """A query row with a NaN gives NaN in that row alone; a key that scores -infinity for
    some rows has no weight in them."""
    from bit_moe_expert_route_gb300 import ops
    q, kp, vp, ks, vs, ln = inputs(B, 400, 20, 8, 2, d, d, [20] * B)
    q[1, 5, 3] = float("nan")
    got = ops.prefix_attention(q, kp, vp, ks, vs, ln)
    bad = torch.zeros(B, 8, dtype=torch.bool, device="cuda")
    bad[1, 5] = True
    assert torch.isnan(got[bad]).all() and torch.isfinite(got[~bad]).all()
    q[1, 5, 3] = 1.0
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    kp[77, 0, 0] = float("-inf")  # every score of this key is -infinity
    o, mag = expected(q, kp, vp, ks, vs, ln)
    check(ops.prefix_attention(q, kp, vp, ks, vs, ln), o, mag)


@gpu
@pytest.mark.parametrize("d", [64, 256])
def test_strided_caches_and_scale(d):
    """K and V interleaved in one buffer; a cache with room for more sequences' positions."""
    from bit_moe_expert_route_gb300 import ops
    B, P, S, Hq, Hkv = 6, 200, 50, 8, 2
    q, _, _, _, _, ln = inputs(B, P, S, Hq, Hkv, d, 3)
    pre = torch.randn(P, 2, Hkv, d, device="cuda").bfloat16()
    suf = torch.randn(B, S + 30, 2, Hkv, d, device="cuda").bfloat16()
    args = (q, pre[:, 0], pre[:, 1], suf[:, :S, 0], suf[:, :S, 1], ln)
    check(ops.prefix_attention(*args, scale=0.25), *expected(*args, scale=0.25))
    B, P = 24, 900  # rows and positions enough for the tensor-memory kernel
    q, _, _, _, _, ln = inputs(B, P, S, Hq, Hkv, d, 3)
    pre = torch.randn(P, 2, Hkv, d, device="cuda").bfloat16()
    suf = torch.randn(B, S + 30, 2, Hkv, d, device="cuda").bfloat16()
    args = (q, pre[:, 0], pre[:, 1], suf[:, :S, 0], suf[:, :S, 1], ln)
    check(ops.prefix_attention(*args, scale=0.25), *expected(*args, scale=0.25))


@gpu
def test_late_large_scores_move_the_reference():
    """Keys planted in several slices give one head scores far above the rest; others stay low."""
    from bit_moe_expert_route_gb300 import ops
    q, kp, vp, ks, vs, ln = inputs(5, 3001, 90, 16, 2, 128, 4, [90] * 5)
    u = q[2, 3].float() / q[2, 3].float().norm()
    for j, c in ((100, 20.0), (1500, 40.0), (2900, 60.0), (2901, 60.5)):
        kp[j, 0] = (c * u).bfloat16()
    ks[2, 80, 0] = (61.0 * u).bfloat16()
    kp[:, 1] -= 30 * q[1, 9].bfloat16() / 20
    check(ops.prefix_attention(q, kp, vp, ks, vs, ln), *expected(q, kp, vp, ks, vs, ln))


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_late_large_scores_move_the_reference_of_many_rows(d):
    """As above with rows enough for the tensor-memory kernel: its output is rescaled
    where it lies, for some rows in some tiles."""
    from bit_moe_expert_route_gb300 import ops
    q, kp, vp, ks, vs, ln = inputs(40, 3001, 20, 16, 2, d, 4, [20] * 40)
    for b, h, step in ((2, 3, 0), (17, 9, 1), (39, 15, 0)):
        u = q[b, h].float() / q[b, h].float().norm()
        for j, c in ((100, 20.0), (700, 28.0), (1500, 40.0), (2900, 60.0), (2901, 60.5)):
            kp[j + step * 60, h // 8] = (c * u).bfloat16()
    check(ops.prefix_attention(q, kp, vp, ks, vs, ln), *expected(q, kp, vp, ks, vs, ln))


@gpu
def test_agrees_with_decode_attention():
    """One sequence: the prefix and its own positions are one cache."""
    from bit_moe_expert_route_gb300 import ops
    q, kp, vp, ks, vs, ln = inputs(1, 500, 60, 16, 2, 256, 6, [60])
    one = ops.decode_attention(q[0], torch.cat([kp, ks[0]]), torch.cat([vp, vs[0]]))
    o, mag = expected(q, kp, vp, ks, vs, ln)
    check(ops.prefix_attention(q, kp, vp, ks, vs, ln), o, mag)
    assert torch.all((one.double() - o[0]).abs() <= 1e-4 * (o[0].abs() + o[0].square().mean().sqrt()))


@gpu
def test_captured_in_a_graph():
    from bit_moe_expert_route_gb300 import ops
    x = inputs(4, 300, 20, 16, 2, 256, 8)
    want = ops.prefix_attention(*x)
    out = torch.empty_like(want)
    ws = torch.empty(ops.lib().moe_prefix_attention_workspace_bytes(4, 300, 20, 16, 2, 256), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.prefix_attention(*x, out=out, ws=ws)
    x[5].zero_()  # the lengths are read when the graph runs
    g.replay()
    torch.cuda.synchronize()
    check(out, *expected(*x))
    assert not torch.equal(out, want)


@pytest.fixture(scope="module")
def L():
    from bit_moe_expert_route_gb300 import build as B
    B.build()
    from bit_moe_expert_route_gb300 import ops
    return ops.lib()


def test_refusals(L):
    buf = np.zeros(1 << 16, np.uint8)
    p = (buf.ctypes.data + 255) // 256 * 256
    vp = ctypes.c_void_p

    def call(q=p, kp=p, vpx=p, ldp=128, ks=p, vs=p, seq=1280, lds=128, lens=p, B=2, P=5, S=10, Hq=4, Hkv=2, d=64, scale=0.0, out=p, ws=p,
             n=1 << 40):
        return L.moe_prefix_attention(vp(q), vp(kp), vp(vpx), ldp, vp(ks), vp(vs), seq, lds, vp(lens), B, P, S, Hq, Hkv, d, scale, vp(out),
                                      vp(ws), n, None)
    for bad in (dict(B=-1), dict(B=65536), dict(P=-1), dict(S=-1), dict(d=96), dict(Hkv=0), dict(Hq=3), dict(Hq=34), dict(ldp=120),
                dict(ldp=132), dict(lds=120), dict(lds=129), dict(seq=-8), dict(seq=1284), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(P=(1 << 28) + 1)):
        assert call(**bad) == -3, bad
    for bad in ("q", "kp", "vpx", "ks", "vs", "lens", "out"):
        assert call(**{bad: None}) == -1, bad
    for bad in ("q", "kp", "vpx", "ks", "vs", "out"):
        assert call(**{bad: p + 8}) == -2, bad
    assert call(lens=p + 2) == -2
    for bad in (dict(ws=None, P=5000), dict(ws=None, B=400), dict(ws=p + 64), dict(n=100), dict(P=5000, n=1000)):
        assert call(**bad) == -4, bad
    assert call(B=0, q=None) == 0
    assert L.moe_prefix_attention_workspace_bytes(2, 5, 10, 4, 2, 64) > 0
    assert L.moe_prefix_attention_workspace_bytes(2, 5, 10, 4, 2, 65) == 0


def test_binding_refuses_wrong_tensors():
    from bit_moe_expert_route_gb300 import ops
    q, k = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        ops.prefix_attention(q, k, k)
    with pytest.raises(ValueError, match="float32"):
        ops.prefix_attention(q.float(), k, k)


@gpu
def test_binding_refuses_unlike_caches():
    from bit_moe_expert_route_gb300 import ops
    q, kp, vp, ks, vs, ln = inputs(2, 5, 3, 4, 2, 64, 0)
    with pytest.raises(ValueError, match="strides"):
        ops.prefix_attention(q, kp, torch.cat([vp, vp], dim=1)[:, :2])
    with pytest.raises(ValueError, match="lens"):
        ops.prefix_attention(q, kp, vp, ks, vs)
    with pytest.raises(ValueError, match="k_suffix"):
        ops.prefix_attention(q, kp, vp, ks[:, :, :1], vs, ln)

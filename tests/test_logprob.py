"""moe_token_logprobs against log_softmax in 64 bits.

Top ids have to be equal: largest logit first, ties to the lower index. Of
the fp32 sums: S goes through at most about 70 sequential adds a thread and 12 in
trees (82 * 2^-24), each weight through a rounded distance of up to 40 natural
units (ex2's argument up to 64: 2^-19 absolute, 1.4e-6 relative) and ex2 (2^-22):
S within 7e-6, so a log probability within 7e-6 plus its last roundings
(2^-23 of up to 40): 2e-5 bounds it. The entropy adds U / S, a mean distance of at most
40 with twice that relative error: 6e-4 in the worst case; 1e-4 holds where the
mean distance is at most 7, as for these inputs.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
INF = float("inf")


def expected(z, k):
    z = z.double()
    lp = torch.log_softmax(z, dim=1)
    p = lp.exp()
    ent = -torch.where(p == 0, torch.zeros_like(p), p * lp).sum(dim=1)
    key = torch.where(torch.isnan(z), torch.full_like(z, -INF), z)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    return lp, ent, order


def check(z, ids, k, r):
    lp, ent, order = expected(z, k)
    assert torch.equal(r.top_ids.long(), order)

    def near(a, b, tol):
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        fin = torch.isfinite(b)
        rest = ~fin & ~torch.isnan(b)
        assert torch.equal(a[rest].double(), b[rest])
        assert torch.all((a.double() - b)[fin].abs() <= tol)
    near(r.top_logprobs, lp.gather(1, order), 2e-5)
    near(r.logprob, lp.gather(1, ids.long()[:, None])[:, 0], 2e-5)
    near(r.entropy, ent, 1e-4)


def inputs(N, V, dtype, seed, ld=None, offset=0):
    """Rows ld elements apart, the first one `offset` elements into its buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or V
    flat = torch.randn(offset + N * ld, generator=g, device="cuda").mul(2.5).to(dtype)
    z = flat.as_strided((N, V), (ld, 1), offset)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    return z, ids


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V,k,ld,offset", [
    (1, 1, 1, None, 0), (1, 1, 0, None, 0), (3, 2, 2, None, 1), (2, 31, 31, 33, 3), (5, 100, 32, None, 0), (1, 5000, 20, None, 0),
    (1, 32000, 5, None, 0), (7, 40001, 32, None, 1), (2, 131072, 20, None, 0), (700, 3001, 8, 3007, 5), (33, 65537, 1, 65539, 7),
    (1300, 513, 4, None, 0), (64, 20000, 0, None, 0), (9, 1024, 32, 1025, 1), (17, 1025, 32, 1025, 1), (2500, 4000, 20, 4001, 3),
    (2433, 8192, 32, None, 0), (5, 300000, 32, 300001, 1)])
def test_matches_64_bits(N, V, k, ld, offset, dtype):
    from bit_moe_expert_route_gb300 import ops
    z, ids = inputs(N, V, dtype, N + V, ld, offset)
    check(z, ids, k, ops.token_logprobs(z, ids, top_k=k))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [37, 9000, 70000])
def test_ties_masks_and_infinities(V, dtype):
    from bit_moe_expert_route_gb300 import ops
    z, ids = inputs(12, V, dtype, V)
    z[0] = 1.25                       # every logit alike
    z[1] = -INF                       # nothing is possible
    z[2] = -INF
    z[2, V - 2] = -3.0                # one token is
    z[3, ::2] = -INF
    z[4, 1::3] = torch.finfo(dtype).min
    z[5] = torch.finfo(dtype).min     # masked by the lowest value throughout
    z[6, V // 2] = INF
    z[7, V // 3] = float("nan")
    z[8, V - 1] += 100                # a late logit far above the rest
    z[9] -= 1000
    z[10] = torch.where(torch.arange(V, device="cuda") % 5 == 0, 2.0, -2.0).to(dtype)  # ties across the k-th place
    z[11, :V - 4] = -INF
    r = ops.token_logprobs(z, ids, top_k=32)
    keep = [i for i in range(12) if i != 1]
    sub = ops.TokenLogprobs(*[t[keep] for t in r])
    check(z[keep], ids[keep], 32, sub)
    assert r.entropy[1] == 0 and r.logprob[1] == -INF and torch.all(r.top_logprobs[1] == -INF)
    assert r.top_ids[1].tolist() == list(range(32))


@gpu
def test_lowest_value_and_infinities_together():
    """The lowest finite value counts beside -infinity."""
    from bit_moe_expert_route_gb300 import ops
    z = torch.full((1, 500), -INF, device="cuda")
    z[0, 100:104] = torch.finfo(torch.float32).min
    r = ops.token_logprobs(z, torch.tensor([102], dtype=torch.int32, device="cuda"), top_k=5)
    assert abs(float(r.logprob[0]) + np.log(4)) < 1e-6 and abs(float(r.entropy[0]) - np.log(4)) < 1e-6
    assert r.top_ids[0].tolist() == [100, 101, 102, 103, 0] and float(r.top_logprobs[0, 4]) == -INF


@gpu
def test_peaked_row_keeps_a_small_entropy():
    """One logit 12 above 999 alike: H = log S - U / S near 0.08, with no cancellation."""
    from bit_moe_expert_route_gb300 import ops
    z = torch.zeros(1, 1000, device="cuda")
    z[0, 700] = 12.0
    ids = torch.tensor([700], dtype=torch.int32, device="cuda")
    r = ops.token_logprobs(z, ids)
    lp, ent, _ = expected(z, 1)
    assert abs(float(r.entropy[0]) - float(ent[0])) <= 2e-6
    assert abs(float(r.logprob[0]) - float(lp[0, 700])) <= 2e-6


@gpu
def test_ids_out_of_range_no_ids_and_no_rows():
    from bit_moe_expert_route_gb300 import ops
    z, ids = inputs(4, 1000, torch.bfloat16, 3)
    ids[1], ids[2] = -1, 1000
    r = ops.token_logprobs(z, ids, top_k=3)
    assert torch.isnan(r.logprob[1:3]).all() and torch.isfinite(r.logprob[[0, 3]]).all()
    r2 = ops.token_logprobs(z, top_k=3)
    assert r2.logprob is None and torch.equal(r2.top_ids, r.top_ids) and torch.equal(r2.entropy, r.entropy)
    r3 = ops.token_logprobs(z[:0], ids[:0], top_k=3)
    assert r3.top_ids.shape == (0, 3) and r3.logprob.shape == (0,)


@pytest.fixture(scope="module")
def L():
    from bit_moe_expert_route_gb300 import build as B
    B.build()
    from bit_moe_expert_route_gb300 import ops
    return ops.lib()


def test_refusals(L):
    buf = np.zeros(4096, np.uint8)
    p = (buf.ctypes.data + 255) // 256 * 256
    vp = ctypes.c_void_p

    def call(z=p, type=1, ld=100, ids=p, N=2, V=100, k=4, lp=p, ent=p, ti=p, tl=p):
        return L.moe_token_logprobs(vp(z), type, ld, vp(ids), N, V, k, vp(lp), vp(ent), vp(ti), vp(tl), None)
    for bad in (dict(type=2), dict(type=-1), dict(N=-1), dict(V=0), dict(V=1 << 30, ld=1 << 30), dict(ld=99), dict(k=-1),
                dict(k=33), dict(V=3), dict(V=31, k=32)):
        assert call(**bad) == -3, bad
    for bad in (dict(z=None), dict(ids=None), dict(lp=None), dict(ti=None), dict(tl=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(z=p + 2), dict(z=p + 1, type=0), dict(ids=p + 2), dict(lp=p + 1), dict(ent=p + 2), dict(ti=p + 2), dict(tl=p + 2)):
        assert call(**bad) == -2, bad
    assert call(N=0, z=None) == 0


def test_binding_refuses_wrong_tensors():
    from bit_moe_expert_route_gb300 import ops
    z = torch.zeros(2, 10)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        ops.token_logprobs(z.half())
    with pytest.raises(ValueError, match="GPU"):
        ops.token_logprobs(z)
    with pytest.raises(ValueError, match="top_k"):
        ops.token_logprobs(z, top_k=11)

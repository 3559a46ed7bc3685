"""moe_add_rmsnorm_q8 against the same formulas in 64 bits.

r = bf16(x + residual), u = r * weight (exact in fp32), q the correctly rounded
quotient u * top / max |u|: the codes have to be equal. The scale's fp32 sum
of squares goes through at most 64 sequential adds a thread, 8 warp sums and
5 shuffle steps, each off by 2^-24 at most: under 80 * 2^-24 / 2 after the root,
plus 4 roundings: 3e-6 relative. values is q * scale rounded to bf16: half a
step of bf16 is 2^-8 of the value at most, and the binade's slack holds the
scale's own 3e-6 in all but a rounding's flip (one more step: 2^-8 (1 + 1e-3)).
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
EPS = 1e-6


def e4m3_round(z):
    lo = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(z / lo) * lo


def expected(x, residual, weight, fmt, eps=EPS):
    r = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    rd, wd = r.double(), weight.double()
    u = rd * wd
    a = u.abs().amax(dim=1, keepdim=True)
    top = 127.0 if fmt == "int8" else 448.0
    z = torch.where(a > 0, u * top / a, torch.zeros_like(u))
    q = torch.round(z) if fmt == "int8" else e4m3_round(z)
    scale = a / top / torch.sqrt(rd.square().mean(dim=1, keepdim=True) + eps)
    return r, q, scale


def check(x, residual, weight, fmt, res, eps=EPS):
    r, q, scale = expected(x, residual, weight, fmt, eps)
    assert torch.equal(res.residual, r)
    assert torch.equal(res.q.float().double(), q)
    assert torch.all((res.scale.double()[:, None] - scale).abs() <= 3e-6 * scale)
    if res.values is not None:
        v = q * scale
        assert torch.all((res.values.double() - v).abs() <= 2.0 ** -8 * 1.001 * v.abs())


def inputs(T, d, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, d + pad, generator=g, device="cuda").mul(0.5).bfloat16()[:, :d]
    res = torch.randn(T, d, generator=g, device="cuda").mul(2).bfloat16()
    w = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16()
    return x, res, w


@gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("T,d,pad", [(1, 8, 0), (3, 64, 8), (5, 200, 0), (1, 2048, 0), (7, 2048, 24), (129, 5120, 64),
                                     (2, 16384, 0), (3000, 1096, 0), (2500, 16384, 8), (20000, 264, 0), (1, 16376, 0)])
def test_matches_64_bits(T, d, pad, fmt):
    from bit_moe_expert_route_gb300 import ops
    x, res, w = inputs(T, d, T + d, pad)
    check(x, res, w, fmt, ops.add_rmsnorm_q8(x, w, residual=res, eps=EPS, fmt=fmt, values=True))
    y = ops.add_rmsnorm_q8(x, w, fmt=fmt, eps=EPS)  # no residual, no bf16 values
    assert y.residual is x and y.values is None
    check(x, None, w, fmt, y)


@gpu
def test_residual_in_place_and_repeat():
    from bit_moe_expert_route_gb300 import ops
    x, res, w = inputs(33, 2048, 5)
    first = ops.add_rmsnorm_q8(x, w, residual=res)
    buf = res.clone()
    y = ops.add_rmsnorm_q8(x, w, residual=buf, residual_out=buf)
    assert y.residual is buf and torch.equal(buf, first.residual)
    assert torch.equal(y.q, first.q) and torch.equal(y.scale, first.scale)


@gpu
def test_ties_round_to_even():
    """A row whose largest |u| is 127 (448) has quotients equal to u: halves are ties."""
    from bit_moe_expert_route_gb300 import ops
    u = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5], device="cuda").bfloat16()[None]
    w = torch.ones(8, device="cuda").bfloat16()
    y = ops.add_rmsnorm_q8(u, w)
    assert y.q[0].tolist() == [127, 0, 2, 2, 0, -2, -2, 64]
    u = torch.tensor([448.0, 17.0, 19.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, -17.0], device="cuda").bfloat16()[None]
    y = ops.add_rmsnorm_q8(u, w, fmt="e4m3")
    assert y.q[0].float().tolist() == [448, 16, 20, 1.0, 1.25, 0, 2.0 ** -8, -16]


@gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_of_zeros_small_and_bad_values(fmt):
    from bit_moe_expert_route_gb300 import ops
    x, _, w = inputs(8, 256, 9)
    x[1] = 0
    x[2, 17] = float("inf")
    x[3, 200] = float("nan")
    x[4] = (x[4].float() * 1e-34).bfloat16()
    x[5] = (x[5].float() * 1e25).bfloat16()  # squares pass the fp32 range
    x[6] = (x[6].float() * 1e17).bfloat16()
    x[7] = (x[7].float() * 1e-37).bfloat16()
    y = ops.add_rmsnorm_q8(x, w, fmt=fmt, values=True, eps=EPS)
    q = y.q.float()
    assert y.scale[1] == 0 and not q[1].any() and not y.values[1].any()
    for bad in (2, 3, 5):
        assert torch.isnan(y.scale[bad]) and not q[bad].any() and torch.isnan(y.values[bad]).all()
    ok = [0, 4, 6]
    check(x[ok], None, w, fmt, ops.NormQ8(y.q[ok], y.scale[ok], x[ok], y.values[ok]))
    w2 = w.clone()
    w2[3] = float("nan")
    assert torch.isnan(ops.add_rmsnorm_q8(x[:1], w2, fmt=fmt).scale).all()
    # weights of 1: u is exact although the row is next to fp32's smallest numbers
    one = torch.ones_like(w)
    assert torch.equal(ops.add_rmsnorm_q8(x[7:], one, fmt=fmt).q.float().double(), expected(x[7:], None, one, fmt)[1])


@gpu
def test_no_rows():
    from bit_moe_expert_route_gb300 import ops
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    y = ops.add_rmsnorm_q8(x, torch.ones(64, device="cuda").bfloat16())
    assert y.q.shape == (0, 64) and y.scale.shape == (0,)


@pytest.fixture(scope="module")
def L():
    from bit_moe_expert_route_gb300 import build as B
    B.build()
    from bit_moe_expert_route_gb300 import ops
    return ops.lib()


def test_refusals(L):
    """Every refusal comes before the device is touched (host memory serves as the pointers)."""
    buf = np.zeros(4096, np.uint8)
    p = (buf.ctypes.data + 255) // 256 * 256
    vp = ctypes.c_void_p

    def call(x=p, ldx=64, res=p, w=p, T=2, d=64, eps=1e-6, fmt=0, ro=p, q=p, s=p, v=None):
        return L.moe_add_rmsnorm_q8(vp(x), ldx, vp(res), vp(w), T, d, eps, fmt, vp(ro), vp(q), vp(s), vp(v), None)
    for bad in (dict(T=-1), dict(d=0), dict(d=12), dict(d=16392, ldx=16392), dict(ldx=56), dict(ldx=68),
                dict(fmt=2), dict(fmt=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf"))):
        assert call(**bad) == -3, bad
    for bad in ("x", "w", "q", "s"):
        assert call(**{bad: None}) == -1, bad
    for bad in (dict(x=p + 2), dict(res=p + 8), dict(w=p + 2), dict(ro=p + 4), dict(q=p + 4), dict(s=p + 2), dict(v=p + 8)):
        assert call(**bad) == -2, bad
    assert call(T=0, x=None) == 0


def test_binding_refuses_wrong_tensors():
    from bit_moe_expert_route_gb300 import ops
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="fmt"):
        ops.add_rmsnorm_q8(x, w, fmt="int4")
    with pytest.raises(ValueError, match="float32"):
        ops.add_rmsnorm_q8(x.float(), w)
    with pytest.raises(ValueError, match="GPU"):
        ops.add_rmsnorm_q8(x, w)

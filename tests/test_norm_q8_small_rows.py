"""moe_add_rmsnorm_q8 on rows of small numbers: every code has to be the correctly rounded one
also where products of row and weight fall below fp32's normal range, or where top / max |u|
passes its end (top = 448: from 1.317e-36 down). The references are in 64 bits, where all of
these are exact.

The scale carries test_norm_q8's 3e-6 and, below the normal range, half a step of 2^-149. The bf16
values are q * scale (exact in 64 bits here) rounded once to fp32 and once to bf16: 2^-24 and 2^-8 of it,
or half a step of fp32's (2^-150) and bf16's (2^-134) numbers below the normal range.
"""
import pytest

import test_norm_q8 as N

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
EPS = 1e-6
SIZES = [1.0, 1e-20, 1.3e-24, 8.4e-25, 8.2e-25, 1e-25, 1e-30, 2e-36, 1.32e-36, 1.31e-36, 1.3e-36, 1.1e-36, 1.01e-36, 9.9e-37, 1e-37,
         1.2e-38, 1e-38, 1e-39, 1e-40, 0.0]


def rows(d, seed, sizes=SIZES):
    """A row of each size: its largest element is the size itself (as bf16)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = torch.tensor(sizes, device="cuda", dtype=torch.float64)[:, None]
    x = ((torch.rand(len(sizes), d, generator=g, device="cuda", dtype=torch.float64) * 1.9 - 0.95) * s)
    x[torch.arange(len(sizes)), torch.randint(0, d, (len(sizes),), generator=g, device="cuda")] = s[:, 0]
    return x.float().to(torch.bfloat16)


def check(x, w, fmt, residual=None):
    from bit_moe_expert_route_gb300 import ops
    y = ops.add_rmsnorm_q8(x, w, residual=residual, fmt=fmt, values=True, eps=EPS)
    r, q, scale = N.expected(x, residual, w, fmt, EPS)
    assert torch.equal(y.residual, r)
    wrong = (y.q.float().double() != q).any(dim=1)
    assert not wrong.any(), f"rows with wrong codes: {wrong.nonzero().flatten().tolist()}"
    assert torch.all((y.scale.double()[:, None] - scale).abs() <= 3e-6 * scale + 2.0 ** -150)
    v = q * y.scale.double()[:, None]
    assert torch.all((y.values.double() - v).abs() <= (2.0 ** -8 + 2.0 ** -23) * v.abs() + 2.0 ** -134 + 2.0 ** -150)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [8, 64, 264, 2048, 5120, 16384])
def test_weights_of_one(d, fmt):
    check(rows(d, d), torch.ones(d, device="cuda").bfloat16(), fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("size", [1.0, 1e-10, 1e-30, 1e-38])
def test_any_weights(size, fmt):
    """Products down to 1e-78, below every fp32 number; with and without a residual."""
    for d in (8, 264, 2048):
        g = torch.Generator(device="cuda").manual_seed(d)
        w = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda", dtype=torch.float64)) * size).float().to(torch.bfloat16)
        check(rows(d, d + 1), w, fmt)
        check(rows(d, d + 2), w, fmt, residual=rows(d, d + 3))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_ties_of_small_rows(fmt):
    """Quotients on borders between two codes, at sizes where no fp32 product is normal."""
    top, ties = (127.0, [0.5, 1.5, 2.5, -0.5, -1.5, 63.5, -62.5]) if fmt == "int8" else (448.0, [17.0, 19.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, -17.0])
    x = torch.tensor([[top] + ties], device="cuda", dtype=torch.float64) * 2.0 ** -100
    w = torch.full((8,), 2.0 ** -60, device="cuda").bfloat16()
    check(x.float().to(torch.bfloat16), w, fmt)


def test_large_elements_beside_weights_of_zero():
    """Elements near bf16's end whose weight is 0 do not count, in a row that is small otherwise."""
    x = rows(264, 5, [1e-25, 1e-37, 1e-39])
    w = torch.ones(264, device="cuda").bfloat16()
    x[:, 7], w[7] = 1e18, 0.0
    check(x, w, "int8")
    check(x, w, "e4m3")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_that_are_not_finite_beside_small_ones(fmt):
    from bit_moe_expert_route_gb300 import ops
    x = rows(264, 6, [1e-37, 1.0, 1e-25, 1e-36])
    x[1, 3] = float("nan")
    x[3, 200] = float("inf")
    y = ops.add_rmsnorm_q8(x, torch.ones(264, device="cuda").bfloat16(), fmt=fmt)
    assert torch.isnan(y.scale[[1, 3]]).all() and not y.q[[1, 3]].float().any()
    assert torch.equal(y.q[[0, 2]].float().double(), N.expected(x[[0, 2]], None, torch.ones_like(x[0]), fmt)[1])

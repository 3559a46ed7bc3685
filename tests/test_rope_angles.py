"""The rotation's angles at far positions and large frequencies, against whole-number arithmetic.

A frequency is a fraction of 24 bits, so position * frequency is exact in whole numbers, and is reduced by
2 pi with 300 bits behind the point. Tolerances are test_qk_norm_rope's: 2^-8 of the value, and 2^-19 of
the pair's magnitudes.
"""
import math

import pytest

torch = pytest.importorskip("torch")

BITS = 300


def two_pi():
    """2 pi in units of 2^-BITS, by Machin's formula."""
    one = 1 << (BITS + 32)

    def arctan_of_inverse(x):
        power = one // x
        total, n, sign = power, 3, -1
        while power:
            power //= x * x
            total += sign * (power // n)
            sign, n = -sign, n + 2
        return total
    return 2 * (16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239)) >> 32


def angle(freq, position, whole=two_pi()):
    """position * freq mod 2 pi, in -pi .. pi, rounded to 64 bits once."""
    num, den = freq.as_integer_ratio()
    left = ((num * position) << BITS) // den % whole
    if 2 * left > whole:
        left -= whole
    return left / (1 << BITS)


def test_whole_numbers():
    assert two_pi() / (1 << BITS) == 2 * math.pi
    assert angle(1.0, 3) == 3.0 and angle(-1.0, 3) == -3.0 and abs(angle(0.5, 7) - (3.5 - 2 * math.pi)) < 1e-15
    assert abs(angle(1.0, 1000) - math.remainder(1000.0, 2 * math.pi)) < 1e-12


FREQS = [1.0, 0.999, 3.0, 64.5, 256.25, 1000.3, 4096.0, 9999.9, 20011.7, 32767.0, 65535.996, -60000.25, 1e-7, 2.0 ** -30, 1e-40, 0.0]


@pytest.mark.gpu
@pytest.mark.parametrize("adjacent", [False, True])
def test_far_positions(adjacent):
    from bit_moe_expert_route_gb300 import ops
    from test_qk_norm_rope import check
    g = torch.Generator(device="cuda").manual_seed(3)
    T, n = 3000, len(FREQS)
    freqs = torch.tensor(FREQS, dtype=torch.float32)
    at = torch.randint(-(1 << 31), 1 << 31, (T,), generator=g, device="cuda").to(torch.int32)
    at[:6] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30])
    at[1000:2000] = 2 ** 31 - 1 - torch.arange(1000, device="cuda", dtype=torch.int32)
    q = torch.randn(T, 2, 2 * n, generator=g, device="cuda").bfloat16()
    got, _ = ops.qk_norm_rope(q, None, ops.Rope(freqs.cuda(), adjacent=adjacent), at)
    turned = torch.tensor([[angle(f, p) for f in freqs.tolist()] for p in at.tolist()], dtype=torch.float64, device="cuda")[:, None]
    ia = torch.arange(n, device="cuda") * (2 if adjacent else 1)
    ib = ia + (1 if adjacent else n)
    a, b = q[..., ia].double(), q[..., ib].double()
    mag = a.abs() + b.abs()
    check(got[..., ia], a * turned.cos() - b * turned.sin(), mag)
    check(got[..., ib], a * turned.sin() + b * turned.cos(), mag)


@pytest.mark.gpu
def test_frequencies_out_of_range_are_nan():
    from bit_moe_expert_route_gb300 import ops
    freqs = torch.tensor([65536.0, -65536.0, 3e38, float("inf"), float("nan"), 65535.996, 0.0, 1.0], device="cuda")
    q = torch.ones(5, 1, 16, dtype=torch.bfloat16, device="cuda")
    got, _ = ops.qk_norm_rope(q, None, ops.Rope(freqs), torch.arange(5, dtype=torch.int32, device="cuda"))
    bad = torch.arange(16, device="cuda") % 8 < 5
    assert torch.isnan(got[..., bad]).all() and torch.isfinite(got[..., ~bad]).all()

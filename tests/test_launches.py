"""What calls launch, on a CUDA runtime that launches nothing (fake_cuda.py)."""
import shutil

import pytest

pytest.importorskip("torch")
if not shutil.which("g++"):
    pytest.skip("the fake runtime needs g++", allow_module_level=True)
import fake_cuda as F

# calls whose kernels use more than 48 KB of shared memory (an opt-in on every device)
LARGE = [("gemm_w8_kernel<64, false>", lambda L: F.gemm(L, 40, 20000, 64)),
         ("gemm_w8_kernel<64, true>", lambda L: F.gemm(L, 40, 20000, 64, type=1)),
         ("gemm_w8_kernel<128, false>", lambda L: F.gemm(L, 100, 20000, 256)),
         ("gemm_w8_kernel<128, true>", lambda L: F.gemm(L, 100, 20000, 256, type=1)),
         ("gemm_w8_kernel<256, false>", lambda L: F.gemm(L, 300, 40000, 2048)),
         ("gemm_w8_kernel<256, true>", lambda L: F.gemm(L, 300, 40000, 2048, type=1)),
         ("prefix_kernel<64, 1>", lambda L: F.prefix(L, 2, 9000, 10, 16, 2, 64)),
         ("prefix_kernel<64, 2>", lambda L: F.prefix(L, 3, 9000, 10, 16, 2, 64)),
         ("prefix_kernel<128, 1>", lambda L: F.prefix(L, 2, 9000, 10, 16, 2, 128)),
         ("prefix_kernel<128, 2>", lambda L: F.prefix(L, 3, 9000, 10, 16, 2, 128)),
         ("prefix_kernel<256, 1>", lambda L: F.prefix(L, 2, 9000, 10, 16, 2, 256)),
         ("prefix_kernel<256, 2>", lambda L: F.prefix(L, 3, 9000, 10, 16, 2, 256)),
         ("prefix_joined_kernel<64>", lambda L: F.prefix(L, 2, 700, 16, 16, 2, 64)),
         ("prefix_joined_kernel<128>", lambda L: F.prefix(L, 2, 700, 16, 16, 2, 128)),
         ("prefix_joined_kernel<256>", lambda L: F.prefix(L, 2, 700, 16, 16, 2, 256)),
         ("prefix_tc_kernel<64>", lambda L: F.prefix(L, 64, 9000, 10, 16, 2, 64)),
         ("prefix_tc_kernel<128>", lambda L: F.prefix(L, 64, 9000, 10, 16, 2, 128)),
         ("prefix_tc_kernel<256>", lambda L: F.prefix(L, 64, 9000, 10, 16, 2, 256)),
         ("gdn_scan_kernel<128, 4>", lambda L: F.scan(L, 100, 1, 2, 128, 128))]


@pytest.mark.parametrize("kernel,call", LARGE, ids=[k for k, _ in LARGE])
def test_every_device_of_a_process(kernel, call):
    """A process that calls on one device and then on others."""
    L = F.lib()
    for dev in (1, 0, 5, 1, 90):
        L.fake_set_device(dev)
        before = L.fake_launches()
        assert call(L) == 0, f"device {dev}"
        new = F.launches(L)[before:]
        assert kernel in [n for n, *_ in new] and all(d == dev for *_, d in new)


@pytest.mark.parametrize("dev,call", [(10 + i, c) for i, (_, c) in enumerate(LARGE)], ids=[k for k, _ in LARGE])
def test_a_failed_opt_in_is_not_kept(dev, call):
    """On a device that no other test uses, and on one past those that are remembered."""
    L = F.lib()
    for d in (dev, 100):
        L.fake_set_device(d)
        L.fake_fail_attributes(1)
        assert call(L) != 0
        assert call(L) == 0


MOST = 2**31 - 1  # tokens and output channels of the 8-bit product


@pytest.mark.parametrize("T,N,K", [(MOST, 1, 16), (1, MOST, 16), (9, MOST, 16), (24, MOST - 10, 16), (40, MOST, 16),
                                   (MOST - 100, 40000, 64), (300, MOST, 1024), (64, MOST - 126, 2048)])
def test_the_products_largest_sizes(T, N, K):
    """Grids cover every size that the interface takes: no sum next to 2^31 wraps."""
    L = F.lib()
    assert L.moe_gemm_w8a8_workspace_bytes(T, N, K) >= 256 and F.gemm(L, T, N, K) == 0
    for name, grid, *_ in F.launches(L):
        if name.startswith("gemm_w8_few"):
            m, nt = (int(x) for x in name.split("<")[1][:-1].split(","))
            assert grid[0] * 16 * m >= N and grid[1] * 8 * nt >= T
        elif name == "widen_kernel":
            assert grid[0] * 256 * 16 >= T * K
        else:
            assert grid[0] == 152


def test_the_other_operators_largest_sizes():
    L = F.lib()
    P = F.P
    for d in (8, 264, 2048, 16384):
        assert L.moe_add_rmsnorm_q8(P, d, P, P, MOST, d, 1e-6, 0, P, P, P, P, None) == 0
    for V in (2, 1000, 100000, 2**30 - 1):
        assert L.moe_token_logprobs(P, 0, V, P, MOST, V, 2, P, P, P, P, None) == 0
    for Pn, S, heads in ((2**28, 2**28, (1024, 1024, 64)), (0, 2**28, (16384, 1024, 64)), (2**28, 0, (16, 1, 256)), (0, 0, (16384, 1024, 256))):
        for B in (1, 65535):
            assert F.prefix(L, B, Pn, S, *heads) == 0, (B, Pn, S, heads)

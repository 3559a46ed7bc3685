"""The library's objects linked with a CUDA runtime that launches nothing (fake_cudart.cpp):
calls through the C ABI without a GPU, and what they would have launched."""
import ctypes
import glob
import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None


def lib():
    """The C ABI on the fake runtime (declared as the real one's), reset."""
    global _lib
    if _lib is None:
        from bit_moe_expert_route_gb300 import build as B
        from bit_moe_expert_route_gb300 import ops
        B.build()
        objs = [os.path.join(B.BUILD_DIR, os.path.basename(s) + ".o") for s in B.sources()]
        if any(not os.path.exists(o) or os.path.getmtime(o) > os.path.getmtime(B.SO) for o in objs):
            B.build(force=True)
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc())))
        inc = [d for d in [os.path.join(cuda, "include")] + glob.glob(os.path.join(cuda, "targets", "*", "include"))
               if os.path.exists(os.path.join(d, "cuda_runtime.h"))]
        so = os.path.join(B.BUILD_DIR, "libmoe_fake_runtime.so")
        r = subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I", inc[0], "-o", so,
                            os.path.join(HERE, "fake_cudart.cpp")] + objs, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        _lib = ctypes.CDLL(so, mode=os.RTLD_LOCAL | os.RTLD_NOW)
        _lib.fake_launch.restype = ctypes.c_char_p
        real = ops.lib()
        for name in ("moe_add_rmsnorm_q8", "moe_gemm_w8a8_workspace_bytes", "moe_gemm_w8a8", "moe_token_logprobs",
                     "moe_prefix_attention_workspace_bytes", "moe_prefix_attention", "moe_gdn_scan_ex"):
            f, g = getattr(_lib, name), getattr(real, name)
            f.argtypes, f.restype = g.argtypes, g.restype
    _lib.fake_reset()
    return _lib


def launches(L):
    """[(kernel with its template arguments, grid (x, y, z), cluster, shared bytes, device)]"""
    out = []
    for i in range(L.fake_launches()):
        v = (ctypes.c_int64 * 7)()
        name = L.fake_launch(i, v).decode()
        name = subprocess.run(["c++filt", name], capture_output=True, text=True).stdout.strip()
        name = re.sub(r"\(anonymous namespace\)::|moe::|^void ", "", name.split("(moe::")[0].split("(GemmW8")[0])
        out.append((re.sub(r"\([a-zA-Z ]+\)", "", name).split("(")[0], tuple(v[:3]), v[5], v[4], v[6]))
    return out


# sizes' arguments with dummy addresses (nothing is read)
P = 1 << 20


def gemm(L, T, N, K, type=0, ws=P):
    n = L.moe_gemm_w8a8_workspace_bytes(T, N, K)
    return L.moe_gemm_w8a8(P, K, P, P, P, T, N, K, type, P, N, ws, n, None)


def prefix(L, B, Pn, S, Hq, Hkv, d, ws=P):
    n = L.moe_prefix_attention_workspace_bytes(B, Pn, S, Hq, Hkv, d)
    return L.moe_prefix_attention(P, P, P, Hkv * d, P, P, S * Hkv * d, Hkv * d, P, B, Pn, S, Hq, Hkv, d, 0.0, P, ws, n, None)


def scan(L, T, Hk, Hv, dk, dv):
    return L.moe_gdn_scan_ex(P, P, P, P, P, T, Hk, Hv, dk, dv, P, P, 0, None)

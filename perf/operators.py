"""The serving operators around the layer: their measured cases, inputs, plain forms and 64-bit definitions.

Four operators, each with cases from the smallest call of a decoding loop to a
prefill or scoring pass:

  norm     residual addition, root-mean-square norm and an 8-bit output with a
           scale per token (ops.add_rmsnorm_q8)
  product  8-bit integer matrix product with scales per token and per output
           channel (ops.gemm_w8a8)
  prefix   decode attention of a batch whose sequences share a prefix
           (ops.prefix_attention)
  logprob  log probabilities of given tokens with the distribution's entropy and
           the top alternatives (ops.token_logprobs)
"""
import math

import torch

own = False

_HEADS = {"16x2x256": (16, 2, 256), "32x8x128": (32, 8, 128), "8x8x64": (8, 8, 64), "12x4x128": (12, 4, 128)}


def listed():
    return [
        # one decoded token's hidden row before a projection
        {"name": "norm one token", "op": "norm", "T": 1, "D": 2048, "fmt": "int8", "values": False, "pad": 0},
        # an uneven batch out of a wider buffer (row stride above the width), 8-bit float output
        {"name": "norm 1000 rows e4m3", "op": "norm", "T": 1000, "D": 5120, "fmt": "e4m3", "values": False, "pad": 64},
        # a prefill chunk whose bf16 values are wanted beside the codes (the expert layer reads them)
        {"name": "norm prefill", "op": "norm", "T": 32768, "D": 2048, "fmt": "int8", "values": True, "pad": 0},
        # one token through a projection
        {"name": "product one token", "op": "product", "T": 1, "N": 4608, "K": 2048, "out": "bf16"},
        # a small batch through an output head, fp32 logits; odd sizes
        {"name": "product head 24 tokens", "op": "product", "T": 24, "N": 100003, "K": 2048, "out": "fp32"},
        # a prefill chunk through a projection
        {"name": "product prefill", "op": "product", "T": 8192, "N": 8192, "K": 2048, "out": "bf16"},
        # two continuations of a short prompt
        {"name": "prefix 2 x 700", "op": "prefix", "B": 2, "P": 700, "S": 16, "heads": "16x2x256"},
        # a few continuations of a document, their own tokens ragged
        {"name": "prefix 8 x 8192", "op": "prefix", "B": 8, "P": 8192, "S": 200, "heads": "32x8x128"},
        # a large batch of answers to one long prompt
        {"name": "prefix 64 x 32768", "op": "prefix", "B": 64, "P": 32768, "S": 512, "heads": "16x2x256"},
        # the sampled token of one sequence
        {"name": "logprob one row", "op": "logprob", "N": 1, "V": 32000, "k": 5, "dtype": "bf16"},
        # a batch of sequences, fp32 logits, as many alternatives as are offered to clients
        {"name": "logprob 48 rows fp32", "op": "logprob", "N": 48, "V": 100003, "k": 20, "dtype": "fp32"},
        # scoring every position of a prompt
        {"name": "logprob 2048 rows", "op": "logprob", "N": 2048, "V": 131072, "k": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "product", "prefix", "logprob"])
    if op == "norm":
        D = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, min(32768, 32768 * 2048 // D))
        return {"op": op, "T": T, "D": D, "fmt": rng.choice(["int8", "e4m3"]), "values": rng.random() < 0.5,
                "pad": 8 * rng.randrange(0, 9)}
    if op == "product":
        T, K = _log(rng, 1, 8192), 16 * _log(rng, 8, 512)
        N = _log(rng, 64, max(64, min(131072, 8192 * 8192 * 2048 // (T * K), (1 << 28) // T, (1 << 29) // K)))
        return {"op": op, "T": T, "N": N, "K": K, "out": rng.choice(["bf16", "fp32"])}
    if op == "prefix":
        heads = rng.choice(sorted(_HEADS))
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "P": _log(rng, 1, 32768) - 1, "S": _log(rng, 1, 512), "heads": heads}
    V = _log(rng, 2, 160000)
    N = _log(rng, 1, min(4096, 2048 * 131072 // V))
    return {"op": op, "N": N, "V": V, "k": rng.randrange(0, min(V, 32) + 1), "dtype": rng.choice(["bf16", "fp32"])}


_EPS = 1e-6


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    s = {"case": case, "op": case["op"]}
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        s["x"] = normal(T, D + case["pad"], std=0.5)[:, :D]  # a block's output: rows of a wider buffer where padded
        s["residual"] = normal(T, D, std=2.0)
        s["weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    elif case["op"] == "product":
        T, N, K = case["T"], case["N"], case["K"]

        def codes(rows):  # rows quantised by their largest value: about 4 standard deviations at 127
            return torch.randn(rows, K, generator=g, device="cuda").mul_(127 / 4).round_().clamp_(-127, 127).to(torch.int8)

        s["a"], s["w"] = codes(T), codes(N)
        s["a_scale"] = torch.rand(T, generator=g, device="cuda") * 0.02 + 0.02
        s["w_scale"] = torch.rand(N, generator=g, device="cuda") * 0.0004 + 0.0004
    elif case["op"] == "prefix":
        Hq, Hkv, d = _HEADS[case["heads"]]
        B, P, S = case["B"], case["P"], case["S"]
        s["q"] = normal(B, Hq, d, std=1.5)
        s["k_prefix"], s["v_prefix"] = normal(P, Hkv, d), normal(P, Hkv, d)
        s["k_suffix"], s["v_suffix"] = normal(B, S, Hkv, d), normal(B, S, Hkv, d)
        lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["lens"] = lens
    else:
        N, V = case["N"], case["V"]
        z = torch.randn(N, V, generator=g, device="cuda").mul_(2.5)
        ids = torch.randint(0, V, (N,), generator=g, device="cuda")
        z[torch.arange(N, device="cuda"), ids] += 6.0 * torch.rand(N, generator=g, device="cuda")  # the tokens that came are likely ones
        s["logits"] = z.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["ids"] = ids.to(torch.int32)
    return s


# ------------------------------------------------------------------ the framework's calls
def _own_norm(s):
    from bit_moe_expert_route_gb300 import ops
    c = s["case"]
    r = ops.add_rmsnorm_q8(s["x"], s["weight"], residual=s["residual"], eps=_EPS, fmt=c["fmt"], values=c["values"])
    return {"codes": r.q, "scale": r.scale, "residual": r.residual, "values": r.values}


def _own_product(s):
    from bit_moe_expert_route_gb300 import ops
    return ops.gemm_w8a8(s["a"], s["a_scale"], s["w"], s["w_scale"],
                         dtype=torch.bfloat16 if s["case"]["out"] == "bf16" else torch.float32)


def _own_prefix(s):
    from bit_moe_expert_route_gb300 import ops
    return ops.prefix_attention(s["q"], s["k_prefix"], s["v_prefix"], s["k_suffix"], s["v_suffix"], s["lens"])


def _own_logprob(s):
    from bit_moe_expert_route_gb300 import ops
    r = ops.token_logprobs(s["logits"], s["ids"], top_k=s["case"]["k"])
    return {"logprob": r.logprob, "entropy": r.entropy, "top_ids": r.top_ids, "top_logprobs": r.top_logprobs}


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    c, w = s["case"], s["weight"].float()
    r = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    u = r.float() * w  # exact: two 8-bit significands
    rms = (r.float().square().mean(dim=1) + _EPS).sqrt()
    a = u.abs().amax(dim=1)
    # codes next to a border between two of them: the quotient in 64 bits
    if c["fmt"] == "int8":
        z = (u.double() * 127.0 / a.double()[:, None]).round()
        scale, codes = a / 127.0 / rms, z.to(torch.int8)
    else:
        z = (u.double() * 448.0 / a.double()[:, None]).clamp(-448.0, 448.0)
        scale, codes = a / 448.0 / rms, _e4m3(z).float().to(torch.float8_e4m3fn)
    values = (codes.float() * scale[:, None]).to(torch.bfloat16) if c["values"] else None
    return {"codes": codes, "scale": scale, "residual": r, "values": values}


def _e4m3(z):
    """z (64 bits, |z| <= 448) rounded to the nearest 8-bit float of 4 exponent and 3 fraction bits, ties to even."""
    e = torch.frexp(z).exponent.clamp(min=-5) - 1  # floor(log2 |z|), at least the subnormals' -6
    step = torch.ldexp(torch.ones_like(z), e - 3)
    return (z / step).round() * step


def _plain_product(s):
    out = (s["a"].float() @ s["w"].float().t()) * s["a_scale"][:, None] * s["w_scale"]
    return out.to(torch.bfloat16 if s["case"]["out"] == "bf16" else torch.float32)


def _plain_prefix(s):
    q = s["q"].float()
    B, Hq, d = q.shape
    P, Hkv = s["k_prefix"].shape[:2]
    S, G = s["k_suffix"].shape[1], Hq // Hkv
    rows = q.view(B, Hkv, G, d).permute(1, 0, 2, 3).reshape(Hkv, B * G, d) / math.sqrt(d)
    own_rows = q.view(B, Hkv, G, d) / math.sqrt(d)
    sp = (rows @ s["k_prefix"].float().permute(1, 2, 0)).view(Hkv, B, G, P).transpose(0, 1)
    ss = own_rows @ s["k_suffix"].float().permute(0, 2, 3, 1)  # [B, Hkv, G, S]
    past = torch.arange(S, device=q.device) >= s["lens"][:, None]
    scores = torch.cat([sp, ss.masked_fill(past[:, None, None, :], -math.inf)], dim=3)
    m = scores.amax(dim=3, keepdim=True).clamp(min=-1e30)  # a row with no position keeps a finite reference
    p = (scores - m).exp()
    total = p.sum(dim=3, keepdim=True)
    pp = p[..., :P].transpose(0, 1).reshape(Hkv, B * G, P)
    o = (pp @ s["v_prefix"].float().transpose(0, 1)).view(Hkv, B, G, d).transpose(0, 1)
    o = o + p[..., P:] @ s["v_suffix"].float().transpose(1, 2)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.reshape(B, Hq, d).to(torch.bfloat16)


def _order(z):
    """fp32 values as whole numbers in the same order."""
    i = (z + 0.0).view(torch.int32)
    return (i ^ ((i >> 31) & 0x7FFFFFFF)).long()


def _plain_logprob(s):
    z, k = s["logits"].float(), s["case"]["k"]
    m = z.amax(dim=1, keepdim=True)
    e = (z - m).exp()
    total = e.sum(dim=1)
    log_total = total.log()
    at = z.gather(1, s["ids"].long()[:, None])[:, 0]
    # the likeliest first, equal ones by the lower index: one whole number that is larger for each
    key = _order(z) * (1 << 20) + ((1 << 20) - 1 - torch.arange(z.shape[1], device=z.device))
    top = key.topk(k, dim=1).values
    top_ids = (1 << 20) - 1 - (top & ((1 << 20) - 1))
    return {"logprob": at - m[:, 0] - log_total, "entropy": log_total + (e * (m - z)).sum(dim=1) / total,
            "top_ids": top_ids.to(torch.int32), "top_logprobs": z.gather(1, top_ids) - m - log_total[:, None]}


def run(state):
    if own:
        return {"norm": _own_norm, "product": _own_product, "prefix": _own_prefix, "logprob": _own_logprob}[state["op"]](state)
    return {"norm": _plain_norm, "product": _plain_product, "prefix": _plain_prefix, "logprob": _plain_logprob}[state["op"]](state)


# ------------------------------------------------------------------ what one pass cannot do without
def _expected_len(S):
    return S / 2


def work(case):
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        return {"bytes": T * D * (2 + 2 + 2 + 1 + (2 if case["values"] else 0)) + 2 * D + 4 * T, "flops": 8 * T * D}
    if case["op"] == "product":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": T * K + N * K + 4 * (T + N) + T * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * T * N * K}
    if case["op"] == "prefix":
        Hq, Hkv, d = _HEADS[case["heads"]]
        B, P = case["B"], case["P"]
        own_positions = B * _expected_len(case["S"])  # lengths are even over 0 .. S
        return {"bytes": 4 * Hkv * d * (P + own_positions) + 4 * B * Hq * d + 4 * B,
                "flops": 4 * Hq * d * (B * P + own_positions)}
    N, V, k = case["N"], case["V"], case["k"]
    return {"bytes": N * V * (2 if case["dtype"] == "bf16" else 4) + N * (4 + 8 + 8 * k), "flops": 6 * N * V}


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "product": _exact_product, "prefix": _exact_prefix, "logprob": _exact_logprob}[case["op"]](s)


def _exact_norm(s):
    c = s["case"]
    # the stored residual is a bf16 by definition: the sum's own value is its exact one, and the norm is of the stored row
    total = s["x"].double() + s["residual"].double()
    r = (s["x"].float() + s["residual"].float()).to(torch.bfloat16).double()
    D = r.shape[1]
    u = r * s["weight"].double()
    most = u.abs().max(dim=1, keepdim=True).values
    top = 127.0 if c["fmt"] == "int8" else 448.0
    scale = most / top / torch.sqrt((r * r).sum(dim=1, keepdim=True) / D + _EPS)
    z = u * top / most
    if c["fmt"] == "int8":
        codes = torch.round(z)
    else:
        lo = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
        codes = torch.round(z / lo) * lo
    return {"codes": None if c["fmt"] == "int8" else codes, "scale": scale[:, 0], "residual": total,
            "values": codes * scale if c["values"] else None}


def _exact_product(s):
    a = s["a"].double() * s["a_scale"].double()[:, None]
    return torch.cat([a @ w.double().t() for w in s["w"].split(16384)], dim=1) * s["w_scale"].double()


def _exact_prefix(s):
    q = s["q"].double()
    B, Hq, d = q.shape
    Hkv = s["k_prefix"].shape[1]
    G, lens = Hq // Hkv, s["lens"].tolist()
    out = torch.zeros_like(q)
    for h in range(Hkv):  # one key head and one sequence at a time
        kp, vp = s["k_prefix"][:, h].double(), s["v_prefix"][:, h].double()
        for b in range(B):
            k = torch.cat([kp, s["k_suffix"][b, :lens[b], h].double()])
            v = torch.cat([vp, s["v_suffix"][b, :lens[b], h].double()])
            if len(k):
                out[b, h * G:(h + 1) * G] = torch.softmax(q[b, h * G:(h + 1) * G] @ k.t() * d ** -0.5, dim=1) @ v
    return out


def _exact_logprob(s):
    z, k = s["logits"], s["case"]["k"]
    logprob, entropy, top = [], [], []
    for rows, ids in zip(z.split(64), s["ids"].long().split(64)):
        lp = torch.log_softmax(rows.double(), dim=1)
        logprob.append(lp.gather(1, ids[:, None])[:, 0])
        entropy.append(-(lp.exp() * lp).sum(dim=1))
        top.append(lp.topk(k, dim=1).values)
    return {"logprob": torch.cat(logprob), "entropy": torch.cat(entropy), "top_ids": None, "top_logprobs": torch.cat(top)}

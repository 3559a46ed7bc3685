"""The operators of a paged cache: their measured cases, inputs, plain forms and 64-bit definitions.

Three operators of a server that verifies drafted tokens, each with cases from the
smallest call of a decoding loop to a prefill or the longest cache:

  rope    norms of queries and keys for each head and the position rotation in one
          pass, positions of one axis or several (ops.qk_norm_rope)
  append  keys (with norm and rotation on the way) and values appended to a paged
          cache (ops.append_paged)
  tree    attention of a few new tokens a sequence, a tree of drafted ones, over a
          paged cache (ops.tree_attention)
"""
import math

import torch

own = False

_HEADS = {"16x2x256": (16, 2, 256), "32x8x128": (32, 8, 128), "8x8x64": (8, 8, 64), "12x4x128": (12, 4, 128)}
_EPS = 1e-6
_THETA = 1e6


def listed():
    return [
        # one decoded token: a quarter of each head rotates
        {"name": "rope one token", "op": "rope", "T": 1, "heads": "16x2x256", "rotary": 64, "axes": 1, "cyclic": False,
         "adjacent": False, "norm": True, "far": 40000},
        # patches of images: time, height and width as positions, out of the projection's wider rows
        {"name": "rope 1003 patches", "op": "rope", "T": 1003, "heads": "32x8x128", "rotary": 128, "axes": 3, "cyclic": False,
         "adjacent": False, "norm": True, "far": 4000},
        # a prefill chunk at the end of a long context, no norms
        {"name": "rope far chunk", "op": "rope", "T": 4099, "heads": "12x4x128", "rotary": 128, "axes": 1, "cyclic": False,
         "adjacent": True, "norm": False, "far": 1000000},
        # a prefill batch
        {"name": "rope prefill", "op": "rope", "T": 32768, "heads": "16x2x256", "rotary": 64, "axes": 1, "cyclic": False,
         "adjacent": False, "norm": True, "far": 40000},
        # one decoded token
        {"name": "append one token", "op": "append", "B": 1, "N": 1, "L": 4000, "heads": "16x2x256", "rotary": 64, "page": 16,
         "norm": True, "rows": False},
        # what was accepted of 64 sequences' drafts: paths of their trees, appended again behind one another
        {"name": "append accepted paths", "op": "append", "B": 64, "N": 301, "L": 2000, "heads": "32x8x128", "rotary": 128,
         "page": 64, "norm": True, "rows": True},
        # ragged prompts of a prefill batch
        {"name": "append prompts", "op": "append", "B": 7, "N": 32768, "L": 0, "heads": "16x2x256", "rotary": 64, "page": 32,
         "norm": True, "rows": False},
        # a short draft for one sequence
        {"name": "tree 1 x 5 over 700", "op": "tree", "B": 1, "n": 5, "L": 700, "heads": "16x2x256", "page": 16, "tree": True},
        # ordinary decoding, one token of each of many sequences
        {"name": "tree 64 x 1 over 4096", "op": "tree", "B": 64, "n": 1, "L": 4096, "heads": "32x8x128", "page": 64,
         "tree": False},
        # ragged drafts of short sequences with as many key as query heads
        {"name": "tree 48 x 13 over 1500", "op": "tree", "B": 48, "n": 13, "L": 1500, "heads": "8x8x64", "page": 32,
         "tree": True},
        # drafts over long contexts
        {"name": "tree 8 x 16 over 32768", "op": "tree", "B": 8, "n": 16, "L": 32768, "heads": "16x2x256", "page": 64,
         "tree": True},
        # the widest trees over long contexts
        {"name": "tree 4 x 64 over 50001", "op": "tree", "B": 4, "n": 64, "L": 50001, "heads": "16x2x256", "page": 128,
         "tree": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "tree"])
    heads = rng.choice(sorted(_HEADS))
    Hq, Hkv, d = _HEADS[heads]
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        rotary = rng.choice([r for r in (32, 64, 128, 256) if r <= d])
        axes = rng.choice([1, 1, 3])
        return {"op": op, "T": _log(rng, 1, 32768 * 18 * 256 // ((Hq + Hkv) * d)), "heads": heads, "rotary": rotary,
                "axes": axes, "cyclic": axes > 1 and rng.random() < 0.5, "adjacent": rng.random() < 0.3, "norm": rng.random() < 0.7, "far": _log(rng, 1000, 1000000)}
    if op == "append":
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "N": _log(rng, 1, 32768 * 2 * 256 // (Hkv * d)), "L": _log(rng, 1, 4096) - 1, "heads": heads,
                "rotary": rng.choice([0, 32, d]), "page": page, "norm": rng.random() < 0.6, "rows": rng.random() < 0.3}
    B, n = _log(rng, 1, 64), _log(rng, 1, 64)
    cost = 4 * 64 * 50001 * 16 * 256  # of the listed largest
    most = min(131072, cost // (B * n * Hq * d), 8 * 32768 * 2 * 256 // (B * Hkv * d))
    return {"op": op, "B": B, "n": n, "L": _log(rng, 1, most) - 1, "heads": heads, "page": page, "tree": rng.random() < 0.7}


def _sections(pairs, axes, cyclic):
    """Pairs of each axis: some of time, the rest shared by height and width (in turn with time's: at most a third each)."""
    if axes == 1:
        return (pairs,)
    side = 5 * pairs // 16 if cyclic else 3 * pairs // 8
    return (pairs - 2 * side, side, side)


def _axis_of_pairs(sections, cyclic):
    if not cyclic:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    A, pairs = len(sections), sum(sections)
    return [i % A if i < A * sections[i % A] else 0 for i in range(pairs)]


def _cached(B, L):
    """The sequences' cached positions: L down to about half of it, odd numbers among them."""
    return [L - (L // 2) * b // max(1, B - 1) if B > 1 else L for b in range(B)]


def _news(B, n):
    """New tokens of each sequence: mostly n, some fewer."""
    return [n if b % 4 < 2 else max(1, n - (b % 4) * n // 5) for b in range(B)]


def _split(N, B):
    """N tokens over B sequences, unevenly (some have none where N is small)."""
    cuts = [N * (b * b + b) // (B * B + B) for b in range(B + 1)]
    return [cuts[b + 1] - cuts[b] for b in range(B)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    def weight(d):
        return (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)

    def freqs(r):
        i = torch.arange(0, r, 2, dtype=torch.float64)
        return (_THETA ** (-i / r)).to(torch.float32).cuda()

    def device(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype).cuda()

    Hq, Hkv, d = _HEADS[case["heads"]]
    s = {"case": case, "op": case["op"]}
    if case["op"] == "rope":
        T = case["T"]
        qkv = normal(T, Hq + 2 * Hkv, d, std=1.5)  # one projection's output: queries and keys are views of it
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        s["q_weight"], s["k_weight"] = (weight(d), weight(d)) if case["norm"] else (None, None)
        s["freqs"], s["sections"] = freqs(case["rotary"]), _sections(case["rotary"] // 2, case["axes"], case["cyclic"])
        at = torch.randint(0, case["far"], (case["axes"], T), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = at[0] if case["axes"] == 1 else at
        return s
    B, page, L = case["B"], case["page"], case["L"]
    turn = torch.randperm(B, generator=host).tolist()
    lens = [_cached(B, L)[b] for b in turn]
    news = [(_split(case["N"], B) if case["op"] == "append" else _news(B, case["n"]))[b] for b in turn]
    N = sum(news)
    needed = [-(-(a + b) // page) for a, b in zip(lens, news)]
    width = max(needed) + 1
    order = torch.randperm(sum(needed) + 3, generator=host).tolist()  # pages in no order, a few of them unused
    table, at = torch.full((B, width), -1, dtype=torch.int32), 0
    for b, n in enumerate(needed):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    s["starts"], s["lens"], s["table"] = device(starts), device(lens), table.cuda()
    pool = (len(order), page, Hkv, d)
    if case["op"] == "append":
        most = 2 * N if case["rows"] else N  # the drafts that the accepted ones are rows of
        qkv = normal(most, Hq + 2 * Hkv, d, std=1.5) if most <= 4096 else normal(most, 2 * Hkv, d, std=1.5)
        s["k"], s["v"] = qkv[:, -2 * Hkv:-Hkv], qkv[:, -Hkv:]
        s["k_pages"], s["v_pages"] = torch.zeros(pool, dtype=torch.bfloat16, device="cuda"), torch.zeros(pool, dtype=torch.bfloat16, device="cuda")
        s["rows"] = torch.randperm(most, generator=host)[:N].sort().values.to(torch.int32).cuda() if case["rows"] else None
        s["k_weight"] = weight(d) if case["norm"] else None
        s["freqs"] = freqs(case["rotary"]) if case["rotary"] else None
        return s
    s["q"] = normal(N, Hq, d, std=1.5)
    s["k_pages"], s["v_pages"] = normal(*pool), normal(*pool)
    s["tree"] = None
    if case["tree"]:
        bits = []
        for n in news:  # each token's parent is an earlier one, or the last cached token
            up = (torch.rand(n, generator=host) * torch.arange(1, n + 1)).long().tolist()
            masks = []
            for i, j in enumerate(up):
                masks.append((1 << i) | (masks[j - 1] if j > 0 else 0))
            bits += masks
        s["tree"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in bits], dtype=torch.int64).cuda()
    return s


# ------------------------------------------------------------------ the framework's calls
def _own_rope(s):
    from bit_moe_expert_route_gb300 import ops
    c = s["case"]
    rope = ops.Rope(s["freqs"], s["sections"], c["cyclic"], c["adjacent"])
    q, k = ops.qk_norm_rope(s["q"], s["k"], rope, s["positions"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=_EPS)
    return {"q": q, "k": k}


def _own_append(s):
    from bit_moe_expert_route_gb300 import ops
    cache = ops.PagedCache(s["k_pages"], s["v_pages"], s["table"])
    rope = None if s["freqs"] is None else ops.Rope(s["freqs"])
    ops.append_paged(s["k"], s["v"], cache, s["starts"], s["lens"], rope, k_weight=s["k_weight"], eps=_EPS, rows=s["rows"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_tree(s):
    from bit_moe_expert_route_gb300 import ops
    cache = ops.PagedCache(s["k_pages"], s["v_pages"], s["table"])
    return ops.tree_attention(s["q"], cache, s["starts"], s["lens"], s["tree"])


# ------------------------------------------------------------------ plain forms
def _normed(x, w):
    x = x.float()
    if w is None:
        return x
    return x / ((x * x).mean(dim=-1, keepdim=True) + _EPS).sqrt() * w.float()


def _rotated(y, angle, adjacent):
    """y fp32 [T, H, d] with its first elements rotated by angle (64 bits) [T, pairs]."""
    n = angle.shape[1]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if adjacent:
        a, b = y[..., 0:2 * n:2], y[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = y[..., :n], y[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([turned, y[..., 2 * n:]], dim=-1)


def _plain_rope(s):
    c = s["case"]
    at = s["positions"] if c["axes"] > 1 else s["positions"][None]
    axis = torch.tensor(_axis_of_pairs(s["sections"], c["cyclic"]), device=at.device)
    angle = at[axis].t().double() * s["freqs"].double()
    return {n: _rotated(_normed(s[n], s[n + "_weight"]), angle, c["adjacent"]).to(torch.bfloat16) for n in ("q", "k")}


def _places(s, N):
    """Sequence and position of each new token."""
    t = torch.arange(N, device=s["starts"].device)
    b = torch.searchsorted(s["starts"].long(), t, right=True) - 1
    return b, s["lens"].long()[b] + t - s["starts"].long()[b]


def _plain_append(s):
    c, page = s["case"], s["case"]["page"]
    b, at = _places(s, c["N"])
    k, v = (s["k"], s["v"]) if s["rows"] is None else (s["k"][s["rows"].long()], s["v"][s["rows"].long()])
    y = _normed(k, s["k_weight"])
    if s["freqs"] is not None:
        y = _rotated(y, at[:, None].double() * s["freqs"].double(), False)
    to = s["table"][b, at // page].long()
    s["k_pages"][to, at % page] = y.to(torch.bfloat16)
    s["v_pages"][to, at % page] = v
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_tree(s):
    c, q = s["case"], s["q"].float()
    N, Hq, d = q.shape
    B, width = s["table"].shape
    page, Hkv = s["k_pages"].shape[1:3]
    pages = s["table"].long().clamp(min=0)
    P = width * page
    k, v = (s[n][pages].view(B, P, Hkv, d).permute(0, 2, 1, 3).float() for n in ("k_pages", "v_pages"))  # [B, Hkv, P, d]
    b, place = _places(s, N)
    i = torch.arange(N, device=q.device) - s["starts"].long()[b]
    rows = torch.zeros(B, c["n"], Hq, d, device=q.device)
    rows[b, i] = q
    rows = rows.view(B, c["n"], Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d) / math.sqrt(d)
    seen = torch.zeros(B, c["n"], P, dtype=torch.bool, device=q.device)
    new = torch.arange(P, device=q.device) - s["lens"].long()[b][:, None]  # [N, P] which new token a position is
    if s["tree"] is None:
        attends = new <= i[:, None]
    else:
        attends = (new < 0) | (new < 64) & ((s["tree"][:, None] >> new.clamp(0, 63)) & 1).bool()
    seen[b, i] = attends
    seen = seen[:, None, :, None].expand(B, Hkv, c["n"], Hq // Hkv, P).reshape(B, Hkv, -1, P)
    scores = (rows @ k.transpose(2, 3)).masked_fill(~seen, -math.inf)
    p = (scores - scores.amax(dim=3, keepdim=True).clamp(min=-1e30)).exp()
    o = (p @ v) / p.sum(dim=3, keepdim=True).clamp(min=1e-30)
    o = o.view(B, Hkv, c["n"], Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, c["n"], Hq, d)
    return o[b, i].to(torch.bfloat16)


def run(state):
    if own:
        return {"rope": _own_rope, "append": _own_append, "tree": _own_tree}[state["op"]](state)
    return {"rope": _plain_rope, "append": _plain_append, "tree": _plain_tree}[state["op"]](state)


# ------------------------------------------------------------------ what one pass cannot do without
def work(case):
    Hq, Hkv, d = _HEADS[case["heads"]]
    if case["op"] == "rope":
        T = case["T"]
        return {"bytes": 4 * T * (Hq + Hkv) * d + 4 * T * case["axes"] + (4 * d if case["norm"] else 0) + 2 * case["rotary"],
                "flops": T * (Hq + Hkv) * ((4 * d if case["norm"] else 0) + 3 * case["rotary"])}
    if case["op"] == "append":
        N = case["N"]
        return {"bytes": 8 * N * Hkv * d + 8 * case["B"] + (4 * N if case["rows"] else 0),
                "flops": N * Hkv * ((4 * d if case["norm"] else 0) + 3 * case["rotary"])}
    B = case["B"]
    news, cached = _news(B, case["n"]), _cached(B, case["L"])
    N = sum(news)
    return {"bytes": 4 * Hkv * d * (sum(cached) + N) + 4 * N * Hq * d + 8 * B + (8 * N if case["tree"] else 0),
            "flops": sum(4 * Hq * d * n * (2 * a + n) // 2 for n, a in zip(news, cached))}


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "tree": _exact_tree}[case["op"]](s)


def _turn(x, weight, freq, where, adjacent):
    """One head's rows x [T, d] in 64 bits; where [T, pairs]: each pair's position."""
    x = x.double()
    if weight is not None:
        x = x * torch.rsqrt(x.pow(2).sum(dim=1, keepdim=True) / x.shape[1] + _EPS) * weight.double()
    if freq is None:
        return x
    n = len(freq)
    first = torch.arange(n, device=x.device) * (2 if adjacent else 1)
    second = first + (1 if adjacent else n)
    z = torch.complex(x[:, first], x[:, second]) * torch.polar(torch.ones_like(where), where * freq.double())
    out = x.clone()
    out[:, first], out[:, second] = z.real, z.imag
    return out


def _exact_rope(s):
    c, T = s["case"], s["q"].shape[0]
    at = s["positions"].double().view(c["axes"], T, 1)
    where = at[0].repeat(1, len(s["freqs"]))
    for a in range(1, c["axes"]):
        first, n = sum(s["sections"][:a]), s["sections"][a]
        where[:, slice(a, n * c["axes"], c["axes"]) if c["cyclic"] else slice(first, first + n)] = at[a]
    return {n: torch.stack([_turn(s[n][:, h], s[n + "_weight"], s["freqs"], where, c["adjacent"])
                            for h in range(s[n].shape[1])], dim=1) for n in ("q", "k")}


def _exact_append(s):
    page = s["case"]["page"]
    out = {n: s[n].double() for n in ("k_pages", "v_pages")}
    starts, lens, table = s["starts"].tolist(), s["lens"].tolist(), s["table"].tolist()
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        if n == 0:
            continue
        rows = torch.arange(starts[b], starts[b + 1], device="cuda") if s["rows"] is None else s["rows"][starts[b]:starts[b + 1]].long()
        at = [lens[b] + i for i in range(n)]
        to = torch.tensor([table[b][p // page] for p in at], device="cuda")
        on = torch.tensor([p % page for p in at], device="cuda")
        where = None if s["freqs"] is None else torch.tensor(at, dtype=torch.float64, device="cuda")[:, None].expand(n, len(s["freqs"])).contiguous()
        for h in range(s["k"].shape[1]):
            out["k_pages"][to, on, h] = _turn(s["k"][rows, h], s["k_weight"], s["freqs"], where, False)
            out["v_pages"][to, on, h] = s["v"][rows, h].double()
    return out


def _exact_tree(s):
    page, Hkv, d = s["k_pages"].shape[1:]
    Hq = s["q"].shape[1]
    G = Hq // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    tree = None if s["tree"] is None else s["tree"].tolist()
    for b, L in enumerate(lens):
        t0, n = starts[b], starts[b + 1] - starts[b]
        used = s["table"][b, :-(-(L + n) // page)].long()
        hidden = torch.zeros(n, L + n, dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                hidden[i, L + j] = j > i if tree is None else not tree[t0 + i] >> j & 1
        hidden = hidden.cuda().repeat_interleave(G, dim=0)
        for h in range(Hkv):  # one key head of one sequence at a time
            k, v = (s[m][used][:, :, h].reshape(-1, d)[:L + n].double() for m in ("k_pages", "v_pages"))
            rows = s["q"][t0:t0 + n, h * G:(h + 1) * G].reshape(n * G, d).double()
            p = torch.softmax((rows @ k.t() * d ** -0.5).masked_fill(hidden, -math.inf), dim=1)
            out[t0:t0 + n, h * G:(h + 1) * G] = (p @ v).view(n, G, d)
    return out

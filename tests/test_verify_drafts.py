"""examples/verify_drafts.py: every stage of a step against its own formula on the values that the
stage before gave it, with the tolerances of the operators' tests; and the caches that it leaves."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def verifier(batch, cached, heads, page, room=40):
    from bit_moe_expert_route_gb300.synth import LayerShape
    from verify_drafts import Verifier
    shape = LayerShape(d_model=256, n_experts=32, top_k=4, d_ff=256, d_ff_shared=256)
    return Verifier(batch, cached, room=room, vocab=1000, shape=shape, heads=heads, page=page)


def positions_of(v, b, n):
    p = torch.arange(n, device="cuda")
    return v.cache.table[b].long()[p // v.page], p % v.page


@pytest.mark.parametrize("batch,cached,heads,page", [(1, 0, (16, 2, 64), 16), (3, 70, (8, 2, 128), 8), (9, 700, (16, 2, 256), 64)])
def test_stages_of_a_step(batch, cached, heads, page):
    import test_gemm_w8a8 as G
    import test_norm_q8 as N
    import test_qk_norm_rope as R
    import test_tree_attention as A

    def near(got, ref):  # bf16 outputs: fp32 scales (1.3e-7) and one rounding, half a step at most
        assert torch.all((got.double() - ref).abs() <= (2.0 ** -8 + 2e-7) * ref.abs())
    v = verifier(batch, cached, heads, page)
    (Hq, Hkv, d), n = heads, len(v.TREE)
    drafts = (torch.arange(batch * n, dtype=torch.int32, device="cuda").view(batch, n) * 37) % 1000
    for step in range(2):
        lens = v.lens.tolist()
        before = [t.clone() for t in v.cache[:2]]
        r = v.step(drafts)
        N.check(r["x"], None, v.norms[0], "int8", r["n1"])
        near(r["qkv"].view(batch * n, -1), G.exact(r["n1"].q, r["n1"].scale, *v.w_qkv))
        where = (torch.tensor(lens, device="cuda")[:, None] + v.depths).view(-1)
        assert torch.equal(r["positions"].long(), where)
        R.check(r["q"], *R.expected(r["qkv"][:, :Hq], v.norms[4], 1e-6, v.rope, where[None]))
        # what the attention read: the cache before, and the tree's tokens behind it
        ko, kmag = R.expected(r["qkv"][:, Hq:Hq + Hkv], v.norms[5], 1e-6, v.rope, where[None])
        o, mag = torch.zeros_like(r["att"], dtype=torch.float64), torch.zeros_like(r["att"], dtype=torch.float64)
        masks = v.masks.tolist()
        for b in range(batch):
            at = positions_of(v, b, lens[b])
            t = slice(b * n, b * n + n)
            # (the cache's own keys: within a rounding of the formula's, which stand for them here)
            k = torch.cat([before[0][at].double(), ko[t].to(torch.bfloat16).double()])
            val = torch.cat([before[1][at].double(), r["qkv"][t, Hq + Hkv:].double()])
            seen = torch.ones(n, lens[b] + n, dtype=torch.bool, device="cuda")
            for i in range(n):
                for j in range(n):
                    seen[i, lens[b] + j] = bool(masks[b * n + i] >> j & 1)
            for h in range(Hkv):
                G_ = Hq // Hkv
                rows = r["q"][t, h * G_:(h + 1) * G_].reshape(n * G_, d).double()
                p = torch.softmax((rows @ k[:, h].t() * d ** -0.5).masked_fill(~seen.repeat_interleave(G_, 0), float("-inf")), dim=1)
                o[t, h * G_:(h + 1) * G_] = (p @ val[:, h]).view(n, G_, d)
                mag[t, h * G_:(h + 1) * G_] = (p @ val[:, h].abs()).view(n, G_, d)
        # (a key of the tree may be the neighbouring bf16 of the formula's: a score is off by half a step of it, 2^-8 of a
        # sum of magnitudes below 60 at most, where all are; 7 of the keys)
        err = (r["att"].double() - o).abs()
        assert torch.all(err <= 2.0 ** -8 * o.abs() + (1.1e-3 + 2.0 ** -8 * 7) * mag)
        N.check(r["att"].view(batch * n, -1), None, v.norms[1], "int8", r["n2"])
        near(r["out"], G.exact(r["n2"].q, r["n2"].scale, *v.w_out))
        N.check(r["out"], r["n1"].residual, v.norms[2], "int8", r["n3"])
        assert torch.isfinite(r["moe"]).all()
        N.check(r["moe"], r["n3"].residual, v.norms[3], "int8", r["n4"])
        # the accepted path: from the root, along the likeliest tokens
        top = r["scores"].top_ids.view(batch, n).tolist()
        for b in range(batch):
            path, token = [0], 0
            while True:
                child = [i for i in range(n) if v.TREE[i] == token and int(drafts[b, i]) == top[b][token]]
                if not child:
                    break
                token = child[0]
                path.append(token)
            assert [x for x in r["accepted"][b].tolist() if x >= 0] == path and int(r["count"][b]) == len(path)
            assert int(r["next"][b]) == top[b][token] and int(v.lens[b]) == lens[b] + len(path)
            # the cache: as it was, then the path's keys and values
            at = positions_of(v, b, lens[b] + len(path))
            k, val = v.cache.k_pages[at], v.cache.v_pages[at]
            rows = torch.tensor(path, device="cuda") + b * n
            old = positions_of(v, b, lens[b])
            assert torch.equal(k[:lens[b]], before[0][old]) and torch.equal(val[:lens[b]], before[1][old])
            R.check(k[lens[b]:], ko[rows], kmag[rows])
            assert torch.equal(val[lens[b]:], r["qkv"][rows, Hq + Hkv:])
        # guesses that agree with the scores are accepted next time
        drafts = drafts.clone()
        drafts[:, 0] = r["next"]
        drafts[:, 1] = (drafts[:, 1] + 1) % 1000


def test_drafts_that_the_scores_agree_with_are_accepted():
    """The tokens that a first run finds likeliest, drafted in a second one from the same caches."""
    heads, batch, n = (8, 2, 128), 3, 7
    drafts = torch.arange(batch * n, dtype=torch.int32, device="cuda").view(batch, n)
    for _ in range(4):  # a level of the tree more each time: what is likeliest depends on what comes before
        v = verifier(batch, 50, heads, 16)
        r = v.step(drafts)
        top = r["scores"].top_ids.view(batch, n)
        drafts = drafts.clone()
        for i, p in enumerate(v.TREE):
            if p >= 0 and i in (1, 3, 6):  # one path from the root to a leaf
                drafts[:, i] = top[:, p]
    assert r["count"].tolist() == [4, 4, 4] and torch.all(r["accepted"] == torch.tensor([0, 1, 3, 6], device="cuda"))


def test_a_step_without_room_is_refused():
    v = verifier(2, 10, (8, 2, 64), 16, room=12)
    drafts = torch.zeros(2, 7, dtype=torch.int32, device="cuda")
    v.step(drafts)
    v.step(drafts)
    with pytest.raises(ValueError, match="room for 12"):
        v.step(drafts)

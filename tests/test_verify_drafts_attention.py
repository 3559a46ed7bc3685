"""examples/verify_drafts.py: the attention of a step against the pages as it read them (the step appends the
accepted path over the tree afterwards), with the operator's own tolerance."""
import pytest

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("batch,cached,heads,page", [(1, 0, (16, 2, 64), 16), (3, 70, (8, 2, 128), 8), (9, 700, (16, 2, 256), 64)])
def test_attention_of_a_step(batch, cached, heads, page, monkeypatch):
    import test_tree_attention as A
    from bit_moe_expert_route_gb300 import ops
    from test_verify_drafts import positions_of, verifier
    v = verifier(batch, cached, heads, page)
    (Hq, Hkv, d), n = heads, len(v.TREE)
    calls, attention = [], ops.tree_attention

    def noted(q, cache, starts, lens, tree):
        calls.append([t.clone() for t in (q, cache.k_pages, cache.v_pages, lens)])
        return attention(q, cache, starts, lens, tree)
    monkeypatch.setattr(ops, "tree_attention", noted)
    drafts = (torch.arange(batch * n, dtype=torch.int32, device="cuda").view(batch, n) * 37) % 1000
    for step in range(2):
        r = v.step(drafts)
        (q, kp, vp, lens), = calls
        calls.clear()

        class P:  # what the operator's reference reads
            lens_list, news, starts_list = lens.tolist(), [n] * batch, list(range(0, batch * n + 1, n))
            N = batch * n

            @staticmethod
            def read(b):
                at = positions_of(v, b, P.lens_list[b] + n)
                return kp[at], vp[at]
        P.Hkv = Hkv
        A.check(r["att"], *A.expected(P, q, v.masks))
        drafts = drafts.clone()
        drafts[:, 0] = r["next"]

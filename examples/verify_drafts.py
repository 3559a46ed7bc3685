"""One verification step of drafted tokens: trees of drafts for several sequences, scored at once.

The sequences' keys and values are in one paged cache. A step takes the last accepted token of each
sequence with a tree of drafted ones behind it through a layer (random weights of the layer's
sizes), scores them, accepts the longest path that the scores agree with, and leaves the cache with
the accepted tokens alone:

  residual norm, 8-bit codes         ops.add_rmsnorm_q8
  query, key and value projection    ops.gemm_w8a8
  norms of the heads' queries, rotation   ops.qk_norm_rope
  keys (normed, rotated) and values into the cache   ops.append_paged
  attention over cache + tree        ops.tree_attention
  norm of the heads' outputs         ops.add_rmsnorm_q8
  output projection                  ops.gemm_w8a8
  residual norm (codes and bf16)     ops.add_rmsnorm_q8
  mixture of experts                 ops.DecodeBatch (up to 8 tokens) or ops.Forward
  residual norm                      ops.add_rmsnorm_q8
  output head                        ops.gemm_w8a8, fp32 logits
  scores                             ops.token_logprobs
  accepted paths again, behind one another   ops.append_paged (rows)

Run:  python examples/verify_drafts.py [--batch 4] [--cached 4000] [--steps 3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_moe_expert_route_gb300 import ops, synth  # noqa: E402
from bit_moe_expert_route_gb300.synth import LayerShape  # noqa: E402
from score_continuations import quantised  # noqa: E402


class Verifier:
    """The paged cache of some sequences, with `cached` positions each to begin with, and the weights
    of one layer and the output head."""

    # token 0 is the sequence's last accepted one; two guesses of the next, and so on
    TREE = (-1, 0, 0, 1, 1, 2, 3)

    def __init__(self, batch: int, cached: int, room: int = 64, vocab: int = 32768,
                 shape: LayerShape = LayerShape(), heads=(16, 2, 256), page: int = 16, seed: int = 0):
        self.batch, self.heads, self.page = batch, heads, page
        Hq, Hkv, d = heads
        D = shape.d_model
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*s, std=1.0):
            return torch.randn(*s, generator=g, device="cuda").mul(std).to(torch.bfloat16)
        self.w_qkv = quantised((Hq + 2 * Hkv) * d, D, g)
        self.w_out = quantised(D, Hq * d, g)
        self.w_head = quantised(vocab, D, g)
        self.norms = [(1 + normal(n, std=0.1)).contiguous() for n in (D, Hq * d, D, D, d, d)]
        self.layer = ops.DeviceLayer(synth.layer_weights(shape, seed), shape)
        self.embedding = normal(vocab, D)
        # every fourth pair of a head turns
        self.rope = ops.Rope(ops.rope_freqs(max(16, d // 4), 1e6))
        width = -(-(cached + room) // page)
        pages = torch.randperm(batch * width, generator=torch.Generator().manual_seed(seed))
        pool = (batch * width, page, Hkv, d)
        self.cache = ops.PagedCache(normal(*pool), normal(*pool), pages.to(torch.int32).view(batch, width).cuda())
        self.lens = torch.full((batch,), cached, dtype=torch.int32, device="cuda")
        self.room, self.used = room, 0  # positions behind `cached`, on the host
        n = len(self.TREE)
        masks, depths = ops.tree_masks(self.TREE)
        self.masks, self.depths = masks.cuda().repeat(batch), depths.cuda()
        self.starts = torch.arange(0, batch * n + 1, n, dtype=torch.int32, device="cuda")
        self.parents = torch.tensor(self.TREE, device="cuda")
        self.experts = ops.DecodeBatch(self.layer, batch * n) if batch * n <= 8 else ops.Forward(self.layer, batch * n)

    def step(self, drafts: torch.Tensor) -> dict:
        """drafts int32 [batch, tree]: each sequence's last accepted token and the drafted ones. Returns
        every intermediate by name; "accepted" int64 [batch, depth + 1] the path's places in the tree (-1
        past its end), "next" int32 [batch] the token that follows it."""
        n, depth = len(self.TREE), int(max(ops.tree_masks(self.TREE)[1]))
        if self.used + n > self.room:
            raise ValueError(f"the caches have room for {self.room} positions, {self.used} are in use and a step needs {n}")
        self.used += depth + 1
        B, (Hq, Hkv, d) = self.batch, self.heads
        N = B * n
        x = self.embedding[drafts.view(-1).long()]
        n1 = ops.add_rmsnorm_q8(x, self.norms[0])
        qkv = ops.gemm_w8a8(n1.q, n1.scale, *self.w_qkv).view(N, Hq + 2 * Hkv, d)
        k, v = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        positions = (self.lens[:, None] + self.depths).view(-1)
        q, _ = ops.qk_norm_rope(qkv[:, :Hq], None, self.rope, positions, q_weight=self.norms[4])
        ops.append_paged(k, v, self.cache, self.starts, self.lens, self.rope, positions, k_weight=self.norms[5])
        att = ops.tree_attention(q, self.cache, self.starts, self.lens, self.masks)
        n2 = ops.add_rmsnorm_q8(att.view(N, Hq * d), self.norms[1])
        out = ops.gemm_w8a8(n2.q, n2.scale, *self.w_out)
        n3 = ops.add_rmsnorm_q8(out, self.norms[2], residual=n1.residual, values=True)
        moe = self.experts(n3.values)
        n4 = ops.add_rmsnorm_q8(moe, self.norms[3], residual=n3.residual)
        logits = ops.gemm_w8a8(n4.q, n4.scale, *self.w_head, dtype=torch.float32)
        scores = ops.token_logprobs(logits, top_k=1)
        # a drafted token is accepted where its parent is and the parent's likeliest token is it
        likeliest = scores.top_ids.view(B, n)
        good = torch.zeros(B, n, dtype=torch.bool, device="cuda")
        good[:, 0] = True
        for i in range(1, n):
            p = self.TREE[i]
            taken = torch.zeros_like(good[:, 0])  # one child of a token at most
            for j in range(1, i):
                if self.TREE[j] == p:
                    taken |= good[:, j]
            good[:, i] = good[:, p] & (likeliest[:, p] == drafts[:, i]) & ~taken
        accepted = torch.full((B, depth + 1), -1, dtype=torch.int64, device="cuda")
        for t in range(depth + 1):
            at = good & (self.depths == t)
            accepted[:, t] = torch.where(at.any(dim=1), at.int().argmax(dim=1), -1)
        count = good.sum(dim=1).to(torch.int32)
        follows = likeliest.gather(1, accepted.gather(1, (count - 1).long()[:, None]))[:, 0]
        # the accepted paths' keys and values once more, at the places that they keep
        ends = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), count.cumsum(0).to(torch.int32)])
        rows = torch.full((B * (depth + 1),), -1, dtype=torch.int32, device="cuda")
        to = (ends[:-1, None] + torch.arange(depth + 1, device="cuda"))[accepted >= 0]
        rows[to.long()] = (accepted + n * torch.arange(B, device="cuda")[:, None])[accepted >= 0].to(torch.int32)
        ops.append_paged(k, v, self.cache, ends, self.lens, self.rope, k_weight=self.norms[5], rows=rows)
        self.lens += count
        return dict(x=x, n1=n1, qkv=qkv, q=q, positions=positions, att=att, n2=n2, out=out, n3=n3, moe=moe, n4=n4, logits=logits,
                    scores=scores, accepted=accepted, count=count, next=follows)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--cached", type=int, default=4000)
    ap.add_argument("--steps", type=int, default=3)
    a = ap.parse_args()
    v = Verifier(a.batch, a.cached, room=7 + 5 * a.steps)
    vocab, n = v.embedding.shape[0], len(v.TREE)
    last = torch.arange(a.batch, dtype=torch.int32, device="cuda")
    for i in range(a.steps):
        # (a drafting model's guesses; here any)
        drafts = (last[:, None] * 31 + torch.arange(n, device="cuda", dtype=torch.int32) * 17 + i) % vocab
        drafts[:, 0] = last
        s = v.step(drafts)
        last = s["next"]
        print(f"step {i}: accepted {s['count'].tolist()} tokens, next {last.tolist()}")
    print(f"positions in the caches: {v.lens.tolist()}")


if __name__ == "__main__":
    main()

"""One decode step of several continuations of one prompt, scored.

The prompt's keys and values are held once; every continuation has a small cache of its
own positions. A step takes one token of each through a layer (random weights of the
layer's sizes) and scores the next token that each continuation wants:

  residual norm, 8-bit codes        ops.add_rmsnorm_q8
  query, key and value projection   ops.gemm_w8a8
  attention over prompt + own       ops.prefix_attention
  norm of the heads' outputs        ops.add_rmsnorm_q8
  output projection                 ops.gemm_w8a8
  residual norm (codes and bf16)    ops.add_rmsnorm_q8
  mixture of experts                ops.DecodeBatch (up to 8 continuations) or ops.Forward
  residual norm                     ops.add_rmsnorm_q8
  output head                       ops.gemm_w8a8, fp32 logits
  scores                            ops.token_logprobs

Run:  python examples/score_continuations.py [--batch 8] [--prompt 8192] [--steps 3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_moe_expert_route_gb300 import ops, synth  # noqa: E402
from bit_moe_expert_route_gb300.synth import LayerShape  # noqa: E402


def quantised(rows: int, cols: int, g: torch.Generator):
    """A random weight matrix in 8 bits with a scale per output channel."""
    w = torch.randn(rows, cols, generator=g, device="cuda")
    scale = w.abs().amax(dim=1) / 127
    return (w / scale[:, None]).round().to(torch.int8), scale * cols ** -0.5


class Continuations:
    """A prompt's keys and values, the continuations' caches, and the weights of one layer and
    the output head."""

    def __init__(self, batch: int, prompt: int, room: int = 64, vocab: int = 32768,
                 shape: LayerShape = LayerShape(), heads=(16, 2, 256), seed: int = 0):
        self.batch, self.room, self.heads = batch, room, heads
        Hq, Hkv, d = heads
        D = shape.d_model
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*s, std=1.0):
            return torch.randn(*s, generator=g, device="cuda").mul(std).to(torch.bfloat16)
        self.w_qkv = quantised((Hq + 2 * Hkv) * d, D, g)
        self.w_out = quantised(D, Hq * d, g)
        self.w_head = quantised(vocab, D, g)
        self.norms = [(1 + normal(n, std=0.1)).contiguous() for n in (D, Hq * d, D, D)]
        self.layer = ops.DeviceLayer(synth.layer_weights(shape, seed), shape)
        small = batch <= 8
        self.experts = ops.DecodeBatch(self.layer, batch) if small else ops.Forward(self.layer, batch)
        self.k_prompt, self.v_prompt = normal(prompt, Hkv, d), normal(prompt, Hkv, d)
        self.k_own = torch.zeros(batch, room, Hkv, d, dtype=torch.bfloat16, device="cuda")
        self.v_own = torch.zeros_like(self.k_own)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.steps = 0  # taken: the positions in use, on the host
        self.embedding = normal(vocab, D)
        self.rows = torch.arange(batch, device="cuda")

    def step(self, tokens: torch.Tensor, wanted: torch.Tensor, top_k: int = 5) -> dict:
        """One token of every continuation (int32 [batch]); scores the tokens that come next
        (`wanted`). Returns every intermediate by name, the scores as "scores". `room` steps at
        most."""
        if self.steps >= self.room:
            raise ValueError(f"the continuations' caches hold {self.room} positions, all in use")
        self.steps += 1
        B, (Hq, Hkv, d) = self.batch, self.heads
        x = self.embedding[tokens.long()]
        n1 = ops.add_rmsnorm_q8(x, self.norms[0])
        qkv = ops.gemm_w8a8(n1.q, n1.scale, *self.w_qkv)
        q, k, v = qkv.view(B, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], dim=1)
        at = self.lens.long()
        self.k_own[self.rows, at], self.v_own[self.rows, at] = k, v
        self.lens += 1
        att = ops.prefix_attention(q.contiguous(), self.k_prompt, self.v_prompt, self.k_own, self.v_own,
                                   self.lens)
        n2 = ops.add_rmsnorm_q8(att.view(B, Hq * d), self.norms[1])
        out = ops.gemm_w8a8(n2.q, n2.scale, *self.w_out)
        n3 = ops.add_rmsnorm_q8(out, self.norms[2], residual=n1.residual, values=True)
        moe = self.experts(n3.values)
        n4 = ops.add_rmsnorm_q8(moe, self.norms[3], residual=n3.residual)
        logits = ops.gemm_w8a8(n4.q, n4.scale, *self.w_head, dtype=torch.float32)
        scores = ops.token_logprobs(logits, wanted, top_k=top_k)
        return dict(x=x, n1=n1, qkv=qkv, att=att, n2=n2, out=out, n3=n3, moe=moe, n4=n4,
                    logits=logits, scores=scores)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=3)
    a = ap.parse_args()
    c = Continuations(a.batch, a.prompt, room=a.steps)
    vocab = c.embedding.shape[0]
    tokens = torch.arange(a.batch, dtype=torch.int32, device="cuda")
    total = torch.zeros(a.batch, device="cuda")
    for i in range(a.steps):
        wanted = (tokens * 7 + 13 * i) % vocab
        s = c.step(tokens, wanted)["scores"]
        total += s.logprob
        tokens = s.top_ids[:, 0].contiguous()  # greedy: the likeliest token goes on
        print(f"step {i}: entropy {s.entropy.mean():.3f} nats, likeliest {s.top_logprobs[:, 0].mean():.3f}")
    best = int(total.argmax())
    print(f"best continuation {best}: log probability {total[best]:.3f}")


if __name__ == "__main__":
    main()

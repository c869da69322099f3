"""Serving steps with drafted trees over a paged cache, on the GPU throughout:

  cache slots for the tree's nodes -> their keys and values, turned by their
  depth, into the slots -> attention of the nodes over the sequence and their
  own branches -> logits adjusted for repetition -> verification of the tree ->
  the accepted path's cache entries moved together -> lengths for the next step.

  python examples/serve_tree.py [--requests 32] [--layers 2] [--vocab 32000] [--steps 3]

The model is two projections and an embedding with random weights; a server has
its own.  Drafts are the target's own top tokens of the step before, so some of
them are accepted.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import speculative_decoding_verification_60_gb300 as sv  # noqa: E402
import synth  # noqa: E402


class Model:
    """Embedding, a query-key-value projection and an output projection for every layer, and the head."""

    def __init__(self, layers, heads, kv_heads, dim, vocab, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        wide = heads * dim

        def weights(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[0] ** -0.5).bfloat16()

        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.embed = torch.randn(vocab, wide, generator=g, device=device).bfloat16()
        self.qkv = [weights(wide, wide + 2 * kv_heads * dim) for _ in range(layers)]
        self.mix = [weights(wide, wide) for _ in range(layers)]
        self.head = weights(wide, vocab)
        self.inv_freq = 10000.0 ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float32) / dim)


class Server:
    """The paged cache of every layer, its bookkeeping and the tokens so far."""

    def __init__(self, model, B, page, max_blocks, parent, device, history=256):
        self.model, self.page, self.device = model, page, device
        self.parent = torch.as_tensor(parent, dtype=torch.int32, device=device)
        depth = [0]
        for p in list(parent)[1:]:
            depth.append(depth[p] + 1)
        self.depth, self.max_depth = torch.tensor(depth, dtype=torch.int32, device=device), max(depth)
        self.nodes = len(depth)
        i32 = dict(dtype=torch.int32, device=device)
        self.lens, self.held = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.table = torch.full((B, max_blocks), -1, **i32)
        self.free, self.free_count = torch.arange(B * max_blocks, **i32), torch.tensor([B * max_blocks], **i32)
        self.accepted = None
        shape = (B * max_blocks, page, model.kv_heads, model.dim)
        self.caches = [[torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)] for _ in model.qkv]
        # tokens so far; what has no place there goes into one more column, which nobody reads
        self.tokens, self.said = torch.zeros(B, history + 1, **i32), torch.zeros(B, **i32)
        self.history = self.tokens[:, :history]
        self.errors = []

    def step(self, tokens, repetition=1.1, temperature=0.0, seed=0):
        """tokens [B, nodes]: every request's tree, node 0 its last token.  Returns the verification and the logits."""
        m, B, N = self.model, tokens.shape[0], self.nodes
        if self.accepted is None:  # the first root; later ones are remembered when they are emitted
            self.remember(tokens[:, :1], torch.ones_like(self.said))
        slots = sv.advance_blocks(self.lens, torch.full_like(self.lens, N), self.table, self.held, self.free,
                                  self.free_count, self.page, B * N, accepted_len=self.accepted)
        self.lens, self.held, self.free_count = slots["seq_lens"], slots["held"], slots["free_count"]
        positions = (self.lens[:, None] + self.depth).reshape(-1)  # a node's depth, not its place, turns it
        x = m.embed[tokens.long()].reshape(B * N, -1)
        for (k_cache, v_cache), qkv, mix in zip(self.caches, m.qkv, m.mix):
            split = (x @ qkv).view(B * N, m.heads + 2 * m.kv_heads, m.dim)
            q, k, v = split.split([m.heads, m.kv_heads, m.kv_heads], 1)
            turned = sv.append_kv(q, k, v, positions, slots["slots"], k_cache, v_cache, m.inv_freq)
            seen = sv.tree_attention(turned["q"].view(B, N, m.heads, m.dim), k_cache, v_cache, self.table, self.lens,
                                     parent=self.parent)
            x = torch.nn.functional.rms_norm(x + seen["out"].view(B * N, -1) @ mix, x.shape[-1:])
            self.errors += [turned["dev_error"], seen["dev_error"]]
        logits = (x @ m.head).view(B, N, -1)
        adjusted = sv.adjust_logits(logits, history=self.history, history_lens=self.said, drafted=tokens,
                                    parent=self.parent, repetition=torch.full((B,), repetition, device=self.device))
        verified = sv.verify_tree(adjusted["logits"], logits, tokens, self.parent, self.max_depth, temperature, seed=seed,
                                  child_mode=sv.CHILD_DETERMINISTIC)
        self.accepted = verified["accepted_len"]
        kept = sv.keep_path([c for both in self.caches for c in both], verified["path_nodes"], self.accepted, self.lens,
                            self.table)
        self.errors += [slots["dev_error"], adjusted["dev_error"], verified["dev_error"], kept["dev_error"]]
        self.remember(verified["out_tokens"], self.accepted + 1)
        return verified, adjusted["logits"]

    def remember(self, tokens, counts):
        """The first counts[b] of tokens[b] join the history, as far as there is room."""
        most = self.history.shape[1]
        i = torch.arange(tokens.shape[1], device=self.device)
        at = torch.where(i < counts[:, None], self.said[:, None] + i, most).clamp_(max=most)
        self.tokens.scatter_(1, at.long(), tokens)
        self.said = torch.clamp(self.said + counts, max=most)

    def drafts(self, verified, logits):
        """The next trees: the last emitted token, and below every node the best tokens of the row that emitted it."""
        B = logits.shape[0]
        last = verified["out_tokens"].gather(1, self.accepted[:, None].long())
        row = verified["path_nodes"].gather(1, self.accepted[:, None].long()).long()
        best = logits.gather(1, row[:, :, None].expand(B, 1, logits.shape[2])).topk(self.nodes - 1, dim=2).indices[:, 0]
        return torch.cat([last, best.to(torch.int32)], 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=3)
    args = ap.parse_args()
    dev = torch.device("cuda")
    parent = synth.pruned_tree()  # the 60 best nodes of a tree of depth 5
    model = Model(args.layers, 16, 4, 64, args.vocab, dev)
    server = Server(model, args.requests, 16, 64, parent, dev)
    tokens = synth.uniform_tokens((args.requests, len(parent)), args.vocab, 7).to(dev)
    for i in range(args.steps):
        verified, logits = server.step(tokens, seed=i)
        tokens = server.drafts(verified, logits)
        print(f"step {i}: {float(verified['accepted_len'].float().mean()):.2f} nodes accepted, "
              f"{int(server.lens.sum())} tokens in the cache before it, {int(server.held.sum())} blocks")
    assert not any(int(e) for e in server.errors)


if __name__ == "__main__":
    main()

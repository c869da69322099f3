"""One serving step with online training of the draft model, on the GPU
throughout:

  verify the drafts -> score what was emitted (log probabilities with the
  target's top alternatives) -> give the next step's tokens their cache slots
  -> distil the draft from those alternatives (loss and gradient).

  python examples/serve_and_distill.py [--requests 64] [--drafts 4] [--vocab 128256] [--steps 3]

Logits are synthetic; a server has them from its two models, and hands
`grad` to the draft model's backward pass.
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


class Cache:
    """The paged cache's bookkeeping: lengths, block table and free list."""

    def __init__(self, B, page, max_blocks, blocks, device):
        i32 = dict(dtype=torch.int32, device=device)
        self.page = page
        self.seq_lens, self.held = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.table = torch.full((B, max_blocks), -1, **i32)
        self.free = torch.arange(blocks, **i32)
        self.free_count = torch.tensor([blocks], **i32)

    def advance(self, new_tokens, max_tokens, accepted_len=None):
        out = sv.advance_blocks(self.seq_lens, new_tokens, self.table, self.held, self.free, self.free_count, self.page,
                                max_tokens, accepted_len=accepted_len)
        self.seq_lens, self.held, self.free_count = out["seq_lens"], out["held"], out["free_count"]
        return out


def step(target, draft, draft_tokens, cache, new_tokens, temperature=1.0, top_p=1.0, seed=0, top_k=20, request_ids=None,
         positions=None):
    """target [B, k+1, V], draft [B, k, V], draft_tokens [B, k].  Returns the
    verification's, the scores', the slots' and the distillation's outputs."""
    B, k, _ = draft.shape
    verified = sv.verify_linear(target, draft, draft_tokens, temperature, top_p, seed, request_ids=request_ids,
                                positions=positions)
    accepted = verified["accepted_len"]
    # every emitted token is scored by the row that emitted it; the -1 entries are skipped
    scores = sv.token_logprobs(target, verified["out_tokens"], top_k=top_k)
    slots = cache.advance(new_tokens, B * (k + 1), accepted_len=accepted)
    # The draft's rows up to the first rejection, where the target has spoken.
    weights = (torch.arange(k, device=draft.device) <= accepted[:, None]).float()
    distilled = sv.distill_topk(draft, scores["top_ids"][:, :k].contiguous(),
                                scores["top_logprobs"][:, :k].contiguous(), weights=weights, tail=sv.TAIL_BUCKET)
    return verified, scores, slots, distilled


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--vocab", type=int, default=128256)
    ap.add_argument("--steps", type=int, default=3)
    args = ap.parse_args()
    B, k, V, dev = args.requests, args.drafts, args.vocab, torch.device("cuda")
    cache = Cache(B, 16, 64, B * 64, dev)
    new = torch.full((B,), k + 1, dtype=torch.int32, device=dev)
    cache.advance(new, B * (k + 1))  # the first step's slots: nothing is verified yet
    for i in range(args.steps):
        target, draft = synth.linear_logits(B, k, V, "bf16", data_seed=100 + i, device=dev)
        drafts = sv.sample_rows(draft.view(B * k, V), 1.0, seed=i)["out_tokens"].view(B, k)
        verified, scores, slots, distilled = step(target, draft, drafts, cache, new, seed=i)
        emitted = verified["out_tokens"] >= 0
        print(f"step {i}: {float(verified['accepted_len'].float().mean()):.2f} drafts accepted, "
              f"log probability {float(scores['logprob'][emitted].mean()):.3f}, "
              f"entropy {float(scores['entropy'][emitted].mean()):.3f}, "
              f"cache {int(cache.seq_lens.sum())} tokens in {int(cache.held.sum())} blocks, "
              f"loss {float(distilled['loss'].sum() / (distilled['loss'] != 0).sum().clamp(min=1)):.4f}")
        for out in (verified, scores, slots, distilled):
            assert int(out["dev_error"]) == 0


if __name__ == "__main__":
    main()

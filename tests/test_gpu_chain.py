"""Calls in a row on one stream, each reading what the one before wrote: the
same bits as with a synchronisation after every call."""

import pytest
import torch

import speculative_decoding_verification_60_gb300 as sv

pytestmark = pytest.mark.gpu


def _chain(target, student, tokens, state, K, wait):
    scores = sv.token_logprobs(target, tokens, top_k=K)
    wait()
    loss = sv.distill_topk(student, scores["top_ids"], scores["top_logprobs"], weights=scores["entropy"])
    wait()
    later = sv.distill_topk_backward(student, scores["top_ids"], scores["top_logprobs"], loss["row_stats"], loss["loss"])
    wait()
    both = sv.token_logprobs(later["grad"], tokens, top_k=K)
    wait()
    slots = sv.advance_blocks(state["seq_lens"], scores["rank"].clamp(0, 3).to(torch.int32), state["table"],
                              state["held"], state["free"], state["free_count"], 4, 3 * len(tokens))
    wait()
    return [scores["logprob"], scores["top_ids"], loss["loss"], loss["grad"], both["logprob"], both["top_ids"],
            slots["slots"], slots["held"], slots["dev_error"], loss["dev_error"], scores["dev_error"]]


@pytest.mark.parametrize("R,V,K", [(3, 40003, 5), (40, 20000, 20), (330, 4096, 8), (1300, 1000, 3)])
def test_a_chain_without_waits_gives_the_same(R, V, K):
    g = torch.Generator(device="cuda").manual_seed(R)
    i32 = dict(dtype=torch.int32, device="cuda")
    rounds = []
    for i in range(6):
        target = torch.randn(R, V, generator=g, device="cuda").bfloat16()
        student = torch.randn(R, V, generator=g, device="cuda").bfloat16()
        tokens = torch.randint(-1, V, (R,), generator=g, device="cuda").to(torch.int32)
        rounds.append((target, student, tokens))

    def state():
        return dict(seq_lens=torch.zeros(R, **i32), held=torch.zeros(R, **i32), free=torch.arange(R, **i32),
                    free_count=torch.tensor([R], **i32), table=torch.full((R, 4), -1, **i32))

    want = [_chain(*r, state(), K, torch.cuda.synchronize) for r in rounds]
    states = [state() for _ in rounds]
    torch.cuda.synchronize()
    got = [_chain(*r, s, K, lambda: None) for r, s in zip(rounds, states)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8) if x.dtype.is_floating_point else x,
                               y.view(torch.uint8) if y.dtype.is_floating_point else y)

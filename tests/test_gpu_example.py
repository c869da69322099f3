"""The serving step that runs the calls together (examples/): its outputs
against the calls' references, step after step."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import synth
import vocab_reference as ref

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_and_distill.py")


def _example():
    spec = importlib.util.spec_from_file_location("serve_and_distill", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_of_serving_and_distillation():
    ex = _example()
    B, k, V, K, page = 6, 3, 2001, 10, 4
    dev = torch.device("cuda")
    cache = ex.Cache(B, page, 16, B * 16, dev)
    new = torch.full((B,), k + 1, dtype=torch.int32, device=dev)
    cache.advance(new, B * (k + 1))
    lens = np.zeros(B, np.int64)
    for i in range(4):
        target, draft = synth.linear_logits(B, k, V, "bf16", data_seed=i)
        tokens = synth.uniform_tokens((B, k), V, i)
        tokens[::2] = draft[::2].float().argmax(2).to(torch.int32)
        verified, scores, slots, distilled = ex.step(target.to(dev), draft.to(dev), tokens.to(dev), cache, new, seed=i,
                                                     top_k=K)
        out = verified["out_tokens"].cpu().numpy()
        a = verified["accepted_len"].cpu().numpy()
        want, _ = ref.token_logprobs(target.float().numpy().reshape(-1, V), out.reshape(-1), 1.0, K)
        assert np.array_equal(scores["top_ids"].cpu().numpy().reshape(-1, K), want["top_ids"])
        np.testing.assert_allclose(scores["logprob"].cpu().numpy().reshape(-1), want["logprob"], rtol=1e-5, atol=1e-5)
        lens += a + 1
        assert np.array_equal(cache.seq_lens.cpu().numpy(), lens)
        position = slots["positions"].cpu().numpy().reshape(B, k + 1)
        assert np.array_equal(position, lens[:, None] + np.arange(k + 1))
        slot = slots["slots"].cpu().numpy()
        assert (slot >= 0).all() and len(set(slot.tolist())) == B * (k + 1)
        loss, grad = distilled["loss"].cpu().numpy(), distilled["grad"].float().cpu().numpy()
        for b in range(B):
            for j in range(k):
                if j > a[b]:
                    assert loss[b, j] == 0 and not grad[b, j].any()
                    continue
                ids = want["top_ids"].reshape(B, k + 1, K)[b, j]
                lp = scores["top_logprobs"][b, j].cpu().numpy()
                l, g, scale, err = ref.distill_row(draft[b, j].float().numpy(), ids, lp, 1.0, True)
                assert err == 0 and abs(loss[b, j] - l) <= ref.distill_loss_bound(draft[b, j].float().numpy(), ids, lp, 1.0)
                np.testing.assert_allclose(grad[b, j], g, rtol=2.0 ** -7, atol=1e-6)

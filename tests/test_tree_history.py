"""The history of examples/serve_tree.py: the first root and every emitted token, in order, whatever was rejected beside
it."""

import importlib.util
import os

import numpy as np
import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_tree.py")


def _example():
    spec = importlib.util.spec_from_file_location("serve_tree", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def held(server):
    return [row[:n] for row, n in zip(server.history.tolist(), server.said.tolist())]


def test_what_is_remembered():
    ex, cpu, B, W, most = _example(), torch.device("cpu"), 6, 4, 17
    server = ex.Server(ex.Model(1, 2, 1, 8, 50, cpu), B, 4, 2, [-1, 0, 0], cpu, history=most)
    rng = np.random.default_rng(0)
    plain = [[] for _ in range(B)]
    for step in range(7):  # more than there is room for
        counts = rng.integers(1, W + 1, B)
        counts[0] = 1  # the others are rejected, in the first step too
        tokens = rng.integers(1, 50, (B, W))
        for b in range(B):
            plain[b] = (plain[b] + tokens[b, :counts[b]].tolist())[:most]
        tokens = np.where(np.arange(W) < counts[:, None], tokens, -1)
        server.remember(torch.tensor(tokens, dtype=torch.int32), torch.tensor(counts, dtype=torch.int32))
        assert held(server) == plain


@pytest.mark.gpu
def test_steps():
    """What the adjustment gets ends with the root's token; the list is kept here."""
    ex, dev, B, V = _example(), torch.device("cuda"), 5, 300
    parent = [-1, 0, 0, 1, 1, 2, 3, 6]
    server = ex.Server(ex.Model(2, 4, 2, 64, V, dev), B, 4, 16, parent, dev, history=40)
    tokens = torch.tensor(np.random.default_rng(0).integers(1, V, (B, len(parent))), dtype=torch.int32, device=dev)
    plain = [[t] for t in tokens[:, 0].tolist()]
    got, adjust = [], ex.sv.adjust_logits

    def spy(logits, **kwargs):
        got.append((kwargs["history"].tolist(), kwargs["history_lens"].tolist(), kwargs["drafted"][:, 0].tolist()))
        return adjust(logits, **kwargs)

    ex.sv.adjust_logits = spy
    try:
        for seed in range(4):
            verified, logits = server.step(tokens, seed=seed)
            history, lens, roots = got[-1]
            assert [row[:n] for row, n in zip(history, lens)] == plain
            assert roots == [row[-1] for row in plain]
            new, counts = verified["out_tokens"].tolist(), (verified["accepted_len"] + 1).tolist()
            plain = [row + t[:n] for row, t, n in zip(plain, new, counts)]
            assert held(server) == plain
            tokens = server.drafts(verified, logits)
    finally:
        ex.sv.adjust_logits = adjust
    assert not any(int(e) for e in server.errors)

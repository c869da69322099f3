"""The history of examples/serve_tree.py: every emitted token, in order, whatever was rejected beside it."""

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

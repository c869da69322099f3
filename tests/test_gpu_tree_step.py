"""The calls of a serving step with drafted trees, one after the other and step after step: slots, appended entries,
attention, adjusted logits, verification, kept path (examples/serve_tree.py), against the plain definitions."""

import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "serve_tree.py")


def _example():
    spec = importlib.util.spec_from_file_location("serve_tree", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps():
    """After every step the cache holds, for the accepted path, what a plain cache of that sequence holds; the attention
    of every layer is the definition's on the cache as it was."""
    ex = _example()
    dev = torch.device("cuda")
    B, page, V = 5, 4, 300
    parent = [-1, 0, 0, 1, 1, 2, 3, 6]
    model = ex.Model(2, 4, 2, 64, V, dev)
    server = ex.Server(model, B, page, 16, parent, dev, history=40)
    svp = ex.sv
    seen, calls = [], {}
    for name in ("append_kv", "tree_attention", "adjust_logits"):
        calls[name] = getattr(svp, name)

    def spy(name):
        def call(*args, **kwargs):
            got = calls[name](*args, **kwargs)
            copy = lambda t: t.clone() if torch.is_tensor(t) else t  # noqa: E731
            seen.append((name, [copy(t) for t in args], {k: copy(t) for k, t in kwargs.items()},
                         {k: copy(t) for k, t in got.items()}))
            return got

        return call

    rng = np.random.default_rng(0)
    tokens = torch.tensor(rng.integers(0, V, (B, len(parent))), dtype=torch.int32, device=dev)
    plain = [[[] for _ in range(B)] for _ in range(4)]  # per plane and request: the entries of its sequence
    accepted_at_all = 0
    try:
        for name in calls:
            setattr(svp, name, spy(name))
        for i in range(5):
            seen.clear()
            verified, logits = server.step(tokens, seed=i)
            torch.cuda.synchronize()
            appended = [s for s in seen if s[0] == "append_kv"]
            attended = [s for s in seen if s[0] == "tree_attention"]
            lens = server.lens.cpu().numpy()
            path, acc = verified["path_nodes"].cpu().numpy(), verified["accepted_len"].cpu().numpy()
            accepted_at_all += int(acc.sum())
            # the attention of every layer, on the cache as it was
            for _, args, kwargs, got in attended:
                q, k_cache, v_cache, table, at = [t.cpu() for t in args]
                want, bound = ref.attend(q, k_cache, v_cache, table, at, torch.tensor(parent), None, 64 ** -0.5)
                assert bool(((got["out"].double().cpu() - want).abs() <= bound).all())
            # adjusted logits of one request
            _, args, kwargs, got = [s for s in seen if s[0] == "adjust_logits"][0]
            b, row = i % B, 7
            raw = args[0][b, row].double().cpu().numpy()
            want = ref.adjust(raw, b, row, kwargs["history"].cpu().numpy(), kwargs["history_lens"].cpu().numpy(), None,
                              kwargs["drafted"].cpu().numpy(), parent, kwargs["repetition"].cpu().numpy(), None, None, None,
                              None, None)
            off = np.abs(got["logits"][b, row].double().cpu().numpy() - want)
            assert (off <= np.abs(want) * ref.half_step(torch.bfloat16) * 1.01 + 1e-6).all()
            # the kept path
            for layer, (_, args, kwargs, _) in enumerate(appended):
                k, v, positions = args[1].cpu(), args[2].cpu(), args[3].cpu()
                _, turned, _ = ref.append(None, k, v, positions, args[4].cpu(), args[5].cpu(), args[6].cpu(),
                                          args[7].cpu(), None, None, 0.0, False)
                for b in range(B):
                    assert len(plain[2 * layer][b]) == lens[b]
                    for plane, x in ((2 * layer, turned), (2 * layer + 1, v.double())):
                        plain[plane][b] += [x[b * len(parent) + p] for p in path[b, :acc[b] + 1]]
            table = server.table.cpu().numpy()
            for plane, cache in enumerate(c for both in server.caches for c in both):
                held = cache.cpu()
                for b in range(B):
                    for t, want in enumerate(plain[plane][b]):
                        got = held[table[b, t // page], t % page].double()
                        assert bool(((got - want).abs() <= want.abs() * 2.0**-8 * 1.01 + want.abs().max() * 2.0**-20).all())
            tokens = server.drafts(verified, logits)
    finally:
        for name, call in calls.items():
            setattr(svp, name, call)
    assert accepted_at_all > 0
    assert not any(int(e) for e in server.errors)


def test_steps_in_a_graph():
    """A layer's calls and the kept path, captured and replayed on other inputs."""
    import speculative_decoding_verification_60_gb300 as svp

    dev = torch.device("cuda")
    B, N, H, K, D, page = 3, 6, 4, 2, 64, 8
    g = torch.Generator(device=dev).manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev).bfloat16()  # noqa: E731
    parent = torch.tensor([-1, 0, 0, 1, 2, 3], dtype=torch.int32, device=dev)
    table = torch.randperm(B * 4, generator=g, device=dev).to(torch.int32).view(B, 4)
    lens = torch.tensor([9, 0, 20], dtype=torch.int32, device=dev)
    at = lens[:, None].long() + torch.arange(N, device=dev)
    slots = (table.gather(1, at // page).long() * page + at % page).view(-1)
    positions = (lens[:, None] + torch.tensor([0, 1, 1, 2, 2, 3], device=dev, dtype=torch.int32)).view(-1)
    inv = 10000.0 ** (-torch.arange(0, D, 2, device=dev, dtype=torch.float32) / D)
    path = torch.tensor([[0, 1, 3, 5], [0, 2, 4, -1], [0, -1, -1, -1]], dtype=torch.int32, device=dev)
    acc = torch.tensor([3, 2, 0], dtype=torch.int32, device=dev)
    qkv, caches = rand(B * N, H + 2 * K, D), [rand(B * 4, page, K, D) for _ in range(2)]

    def layer(qkv, caches, outs):
        q, k, v = qkv.split([H, K, K], 1)
        svp.append_kv(q, k, v, positions, slots, *caches, inv, out=outs[0])
        svp.tree_attention(outs[0]["q"].view(B, N, H, D), *caches, table, lens, parent=parent, out=outs[1])
        svp.keep_path(caches, path, acc, lens, table, out=outs[2])

    outs, spare = [{}, {}, {}], [c.clone() for c in caches]
    layer(qkv, spare, outs)
    graph = torch.cuda.CUDAGraph()
    start = [c.clone() for c in caches]
    with torch.cuda.graph(graph):
        layer(qkv, caches, outs)
    for seed in (5, 6):
        g.manual_seed(seed)
        qkv.copy_(rand(B * N, H + 2 * K, D))
        for c, s in zip(caches, start):
            c.copy_(s)
        graph.replay()
        again, eager = [{}, {}, {}], [s.clone() for s in start]
        layer(qkv, eager, again)
        assert torch.equal(outs[1]["out"], again[1]["out"]) and torch.equal(outs[0]["q"], again[0]["q"])
        assert all(torch.equal(c, e) for c, e in zip(caches, eager))
        assert not any(int(o["dev_error"]) for o in outs)


def test_the_example_runs():
    done = subprocess.run([sys.executable, PATH, "--requests", "4", "--vocab", "2000", "--steps", "2"], cwd=ROOT,
                          capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
    assert done.stdout.count("nodes accepted") == 2

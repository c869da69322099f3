"""Caches of more than 2^31 elements: entries at their end, stored, attended to and moved as in a small cache."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("by_head", [False, True])
def test_the_end_of_a_large_cache(by_head):
    import speculative_decoding_verification_60_gb300 as svp

    dev = torch.device("cuda")
    page, heads, dim, B, N = 64, 4, 128, 2, 5
    blocks = 2**31 // (page * heads * dim) + 300  # 4.3 GB each
    shape = (blocks, heads, page, dim) if by_head else (blocks, page, heads, dim)
    small_shape = (8, heads, page, dim) if by_head else (8, page, heads, dim)
    g = torch.Generator(device=dev).manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev).bfloat16()  # noqa: E731
    large, small = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(2)], [rand(*small_shape) for _ in range(2)]
    for x, y in zip(large, small):
        x[-8:] = y
    view = (lambda t: t.transpose(1, 2)) if by_head else (lambda t: t)
    large, small = [view(x) for x in large], [view(x) for x in small]
    near = torch.tensor([[3, 0, 7], [5, 1, 2]], dtype=torch.int32, device=dev)
    far = near + (blocks - 8)
    assert int(far.max()) * page * heads * dim > 2**31
    lens = torch.tensor([120, 70], dtype=torch.int32, device=dev)
    at = lens[:, None].long() + torch.arange(N, device=dev)
    inv = 10000.0 ** (-torch.arange(0, dim, 2, device=dev, dtype=torch.float32) / dim)
    qkv = rand(B * N, 8 + 2 * heads, dim)
    path = torch.tensor([[0, 2, 4], [0, 3, -1]], dtype=torch.int32, device=dev)
    accepted = torch.tensor([2, 1], dtype=torch.int32, device=dev)
    outs = []
    for caches, table in ((large, far), (small, near)):
        slots = (table.gather(1, at // page).long() * page + at % page).view(-1)
        q, k, v = qkv.split([8, heads, heads], 1)
        turned = svp.append_kv(q, k, v, at.view(-1).to(torch.int32), slots, *caches, inv)
        seen = svp.tree_attention(turned["q"].view(B, N, 8, dim), *caches, table, lens)
        kept = svp.keep_path(caches, path, accepted, lens, table)
        assert not any(int(o["dev_error"]) for o in (turned, seen, kept))
        outs.append(seen["out"])
    assert torch.equal(*outs)
    for x, y in zip(large, small):
        assert torch.equal(x[-8:], y)

"""keep_path against a walk over the entries: the same bytes."""

import numpy as np
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu


def _svp():
    import speculative_decoding_verification_60_gb300 as svp

    return svp


def make(B, W, N, page, lens, accepted, seed=0):
    rng = np.random.default_rng(seed)
    lens, accepted = np.resize(lens, B).astype(np.int32), np.resize(accepted, B).astype(np.int32)
    M = -(-(int(lens.max()) + N) // page)
    table = rng.permutation(B * M + 2)[:B * M].reshape(B, M).astype(np.int32)
    path = np.full((B, W), -1, np.int32)
    for b in range(B):
        a = int(np.clip(accepted[b], 0, W - 1))
        path[b, 0] = 0
        path[b, 1:a + 1] = np.sort(rng.permutation(np.arange(1, N))[:a])
    return lens, accepted, table, path, B * M + 2


def run(case, planes, page, heads, dim, dtype, by_head=False, error=0, refused=(), pad=0):
    lens, accepted, table, path, blocks = case
    g = torch.Generator(device="cuda").manual_seed(3)
    shape = (blocks, heads, page, dim + pad) if by_head else (blocks, page, heads, dim + pad)
    if dtype is torch.uint8:
        whole = [torch.randint(0, 255, shape, generator=g, device="cuda", dtype=dtype) for _ in range(planes)]
    else:
        whole = [torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(planes)]
    caches = [w[..., :dim] for w in whole]
    if by_head:
        caches = [c.transpose(1, 2) for c in caches]
    bits = torch.uint8 if dtype is torch.uint8 else torch.int32 if dtype is torch.float32 else torch.int16
    want = [c.cpu().contiguous().view(bits).numpy().copy() for c in caches]
    beyond = [w[..., dim:].clone() for w in whole]
    c = lambda a: torch.as_tensor(a).cuda()  # noqa: E731
    got = _svp().keep_path(caches, c(path), c(accepted), c(lens), c(table))
    assert int(got["dev_error"]) == error
    for x, y in zip(caches, want):
        assert ref.keep(y, path, accepted, lens, table) == list(refused)
        assert np.array_equal(x.cpu().contiguous().view(bits).numpy(), y)
    for w, y in zip(whole, beyond):
        assert torch.equal(w[..., dim:], y)


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("by_head", [False, True])
def test_pages(page, by_head):
    run(make(4, 6, 30, page, [0, 1, 37, 64], [5, 0, 3, 4]), 3, page, 2, 64, torch.bfloat16, by_head)


@pytest.mark.parametrize("dtype,dim,pad", [(torch.float16, 128, 0), (torch.float32, 20, 0), (torch.uint8, 64, 0),
                                           (torch.uint8, 7, 0), (torch.bfloat16, 9, 0), (torch.bfloat16, 64, 2),
                                           (torch.bfloat16, 64, 1)])
def test_types_and_alignments(dtype, dim, pad):
    run(make(3, 5, 12, 16, [10, 30, 5], [4, 2, 3]), 2, 16, 3, dim, dtype, pad=pad)


@pytest.mark.parametrize("W", [1, 2, 9, 40, 300])
def test_long_paths(W):
    """Longer than what a thread has on its way at once; overlapping moves."""
    run(make(2, W, W + 3, 16, [3, 20], [W - 1, W // 2]), 2, 16, 1, 64, torch.bfloat16)


@pytest.mark.parametrize("planes", [1, 255, 256, 257, 600])
def test_planes(planes):
    run(make(2, 4, 10, 4, [3, 2], [3, 1]), planes, 4, 1, 8, torch.bfloat16)


@pytest.mark.parametrize("case,error", [("accepted", 8), ("negative", 8), ("order", 8), ("twice", 8), ("node", 8),
                                        ("end", 8), ("length", 8), ("block", 32), ("negative block", 32)])
def test_refused_requests(case, error):
    made = make(3, 5, 12, 16, [10, 30, 5], [4, 4, 4])
    lens, accepted, table, path, blocks = made
    if case == "accepted":
        accepted[1] = 5
    elif case == "negative":
        accepted[1] = -1
    elif case == "order":
        path[1, 2], path[1, 3] = path[1, 3], path[1, 2]
    elif case == "twice":
        path[1, 3] = path[1, 2]
    elif case == "node":
        path[1, 0] = -1
    elif case == "end":
        path[1, 4] = 40
    elif case == "length":
        lens[1] = -3
    elif case == "block":
        table[1, 30 // 16] = blocks
    else:
        table[1, 30 // 16] = -1
    run(made, 2, 16, 2, 64, torch.bfloat16, error=error, refused=[1])


def test_a_graph():
    lens, accepted, table, path, blocks = make(3, 5, 12, 16, [10, 30, 5], [4, 2, 3])
    caches = [torch.randn(blocks, 16, 2, 64, device="cuda") for _ in range(4)]
    want = [c.cpu().numpy().copy() for c in caches]
    c = lambda a: torch.as_tensor(a).cuda()  # noqa: E731
    args = (c(path), c(accepted), c(lens), c(table))
    spare = [x.clone() for x in caches]
    out = _svp().keep_path(spare, *args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _svp().keep_path(caches, *args, out=out)
    graph.replay()
    for x, y in zip(caches, want):
        ref.keep(y, path, accepted, lens, table)
        assert np.array_equal(x.cpu().numpy(), y)


def test_planes_that_cannot_be_taken():
    lens, accepted, table, path, blocks = make(2, 3, 6, 4, [3, 2], [2, 1])
    c = lambda a: torch.as_tensor(a).cuda()  # noqa: E731
    args = (c(path), c(accepted), c(lens), c(table))
    a = torch.randn(blocks, 4, 2, 64, device="cuda")
    for planes in ([a, a], [a, a[:-1]], [a, a.bfloat16()], [a, torch.empty(blocks, 2, 4, 64, device="cuda").transpose(1, 2)],
                   [a, a.cpu()], []):
        with pytest.raises(ValueError):
            _svp().keep_path(planes, *args)
    with pytest.raises(ValueError, match="overlap"):
        _svp().keep_path([a[:1].expand(blocks, -1, -1, -1)], *args)

"""tree_attention against the definition in 64 bits: types, head layouts, page sizes, lengths from none on, trees,
counts, what lies behind masks, and what is refused."""

import numpy as np
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu


def _svp():
    import speculative_decoding_verification_60_gb300 as svp

    return svp


def make(B, N, heads, kv, dim, page, lens, dtype=torch.bfloat16, form="chain", counts=None, by_head=False, seed=0,
         spare=3, loud=1.0):
    """Inputs on the CPU.  Whatever no node sees holds NaN: blocks of nobody, entries behind a request's last."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = np.resize(np.asarray(lens), B)
    counts = None if counts is None else np.resize(np.asarray(counts), B)
    M = max(1, -(-(int(lens.max()) + N) // page))
    blocks = B * M + spare
    table = torch.tensor(rng.permutation(blocks)[:B * M].reshape(B, M), dtype=torch.int32)
    shape = (blocks, kv, page, dim) if by_head else (blocks, page, kv, dim)
    k = torch.full(shape, float("nan"), dtype=dtype)
    v = torch.full(shape, float("nan"), dtype=dtype)
    if by_head:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    for b in range(B):
        for t in range(int(lens[b]) + (N if counts is None else int(counts[b]))):
            j, i = int(table[b, t // page]), t % page
            k[j, i] = torch.randn(kv, dim, generator=g).mul_(loud).to(dtype)
            v[j, i] = torch.randn(kv, dim, generator=g).to(dtype)
        used = -(-(int(lens[b]) + (N if counts is None else int(counts[b]))) // page)
        table[b, used:] = torch.tensor([-1, 10**9, -(10**9)], dtype=torch.int32).repeat(M)[:M - used]
    if form == "chain":
        parent = None
    elif form == "tree":
        parent = torch.tensor(ref.random_tree(N, 6, rng), dtype=torch.int32)
    else:
        parent = torch.tensor([ref.random_tree(N, 6, rng) for _ in range(B)], dtype=torch.int32)
    q = torch.randn(B, N, heads, dim, generator=g).to(dtype)
    return dict(q=q, k_cache=k, v_cache=v, block_table=table, seq_lens=torch.tensor(lens, dtype=torch.int32),
                parent=parent, n_nodes=None if counts is None else torch.tensor(counts, dtype=torch.int32),
                scale=dim ** -0.5)


def on_gpu(c):
    """The case on the GPU, with the strides that it has here."""

    def move(t):
        if not torch.is_tensor(t):
            return t
        return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)

    return {key: move(t) for key, t in c.items()}


def check(c, got, error=0):
    want, bound = ref.attend(c["q"], c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], c["parent"],
                             c["n_nodes"], c["scale"])
    assert int(got["dev_error"]) == error
    o = got["out"].double().cpu()
    B, N = o.shape[:2]
    for b in range(B):
        n = N if c["n_nodes"] is None else int(c["n_nodes"][b])
        n = N if n < 0 or n > N else n
        w = want[b, :n]
        assert torch.equal(torch.isnan(w), torch.isnan(o[b, :n])), b
        off = (o[b, :n] - w).abs() - bound[b, :n]
        worst = float(torch.nan_to_num(off, nan=-1.0).max()) if n else -1.0
        assert worst <= 0, (b, worst, float((o[b, :n] - w).abs().max()))
        assert bool((o[b, n:] == 7.0).all()), b  # rows behind a request's nodes stay


def run(c, error=0, **more):
    d = on_gpu(c)
    out = dict(out=torch.full(c["q"].shape, 7.0, dtype=c["q"].dtype, device="cuda"))
    got = _svp().tree_attention(**d, out=out, **more)
    check(c, got, error)
    again = _svp().tree_attention(**d)  # the same bits every time
    live = got["out"] != 7.0
    assert torch.equal(torch.nan_to_num(again["out"][live]), torch.nan_to_num(got["out"][live]))
    return got


@pytest.mark.parametrize("lens", [[0], [1], [0, 1, 126, 127, 128, 129], [255, 256, 700]])
@pytest.mark.parametrize("N", [1, 5])
def test_lengths(lens, N):
    run(make(len(lens), N, 4, 2, 64, 16, lens))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv,dim", [(2, 1, 8), (4, 2, 32), (3, 3, 40), (1, 1, 64), (6, 6, 72), (8, 2, 80), (10, 2, 96), (7, 1, 128), (16, 2, 128)])
def test_heads_and_types(dtype, heads, kv, dim):
    run(make(2, 4, heads, kv, dim, 16, [300, 77], dtype))


@pytest.mark.parametrize("page", [1, 3, 8, 24, 48, 64, 128, 192, 256, 1000])
@pytest.mark.parametrize("by_head", [False, True])
def test_pages(page, by_head):
    run(make(2, 3, 4, 2, 128, page, [270, 131], by_head=by_head))


@pytest.mark.parametrize("N", [2, 31, 32, 33, 60, 64, 65, 100, 129, 200])
@pytest.mark.parametrize("form", ["chain", "tree", "dynamic"])
def test_nodes(N, form):
    run(make(2, N, 2, 1, 64, 32, [150, 5], form=form, seed=N))


@pytest.mark.parametrize("heads,N", [(8, 16), (8, 17), (8, 32), (8, 33), (8, 60), (24, 60), (5, 101)])
def test_many_rows_of_a_head(heads, N):
    """From one tile of 128 query rows to a dozen."""
    run(make(1, N, heads, 1, 128, 16, [200], form="tree", seed=heads + N))


@pytest.mark.parametrize("form", ["chain", "dynamic"])
def test_counts(form):
    run(make(7, 20, 4, 2, 64, 16, [100, 0, 0, 129, 128, 300, 5], form=form, counts=[20, 0, 1, 3, 19, 7, 12]))


@pytest.mark.parametrize("N,heads,kv,B", [(3, 8, 8, 30), (1, 16, 2, 100), (40, 8, 2, 20), (9, 48, 2, 12)])
def test_many_requests(N, heads, kv, B):
    """More tiles than there are CTAs: runs that end within items, requests without nodes between."""
    rng = np.random.default_rng(B)
    counts = rng.integers(0, N + 1, B)
    counts[0], counts[1] = N, 0
    lens = rng.integers(0, 900, B)
    lens[2] = 3000
    run(make(B, N, heads, kv, 64, 64, lens, counts=counts, form="dynamic", seed=B))
    run(make(B, N, heads, kv, 64, 64, lens, seed=B + 1))


@pytest.mark.parametrize("form", ["chain", "tree"])
def test_the_largest_draft(form):
    run(make(1, 1024, 2, 2, 64, 64, [70], form=form, seed=13))


@pytest.mark.parametrize("heads,N", [(128, 3), (100, 2), (65, 5), (127, 1)])
def test_many_heads_a_key_head(heads, N):
    run(make(2, N, heads, 1, 64, 16, [140, 3], form="tree", seed=heads))


def test_more_short_requests_than_a_run_keeps_at_hand():
    rng = np.random.default_rng(14)
    run(make(1500, 1, 8, 8, 64, 8, rng.integers(0, 12, 1500), counts=rng.integers(0, 2, 1500), seed=14))


def test_one_long_sequence():
    run(make(1, 2, 2, 1, 64, 64, [9000], seed=5))


def test_lengths_far_apart():
    run(make(6, 2, 2, 2, 64, 16, [3000, 0, 1, 2, 500, 3], seed=6))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scores_that_rise(dtype):
    """Every tile has larger scores than the one before."""
    c = make(1, 3, 4, 1, 64, 16, [900], dtype, seed=7)
    c["q"] = c["q"].abs()
    for t in range(903):
        c["k_cache"][int(c["block_table"][0, t // 16]), t % 16] *= t / 150
        c["k_cache"][int(c["block_table"][0, t // 16]), t % 16].abs_()
    run(c)


def test_loud_scores():
    run(make(2, 5, 4, 2, 128, 16, [500, 40], loud=30.0, seed=8))


def test_a_fused_projection_and_one_buffer_for_keys_and_values():
    c = make(2, 3, 4, 2, 64, 16, [200, 33], seed=9)
    qkv = torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16)
    qkv[:, :, :4] = c["q"]
    c["q"] = qkv[:, :, :4]
    both = torch.stack([c["k_cache"], c["v_cache"]], dim=1)
    d = on_gpu(c)
    d["q"] = qkv.cuda()[:, :, :4]
    gpu = both.cuda()
    d["k_cache"], d["v_cache"] = gpu[:, 0], gpu[:, 1]
    wide = torch.full((2, c["block_table"].shape[1] + 5), -3, dtype=torch.int32, device="cuda")
    wide[:, :-5] = d["block_table"]
    d["block_table"] = wide[:, :-5]
    check(c, _svp().tree_attention(**d))


def test_nan_in_nodes_stays_on_their_branches():
    c = make(2, 12, 4, 2, 64, 16, [130, 50], form="tree", seed=10)
    leaf = 11
    for b, value in ((0, float("nan")), (1, float("inf"))):
        t = int(c["seq_lens"][b]) + leaf
        c["v_cache"][int(c["block_table"][b, t // 16]), t % 16, 1, 5] = value
    t = 50 + 10
    c["k_cache"][int(c["block_table"][1, t // 16]), t % 16] = float("nan")
    run(c)


@pytest.mark.parametrize("case,error", [
    ("negative length", 8), ("too long", 8), ("count", 8), ("negative count", 8), ("root", 4), ("parent", 4),
    ("block", 32), ("negative block", 32), ("shared tree", 4)])
def test_refused_requests(case, error):
    """Zeros for the refused request, the others as ever."""
    c = make(3, 6, 4, 2, 64, 16, [40, 100, 20], form="tree" if case == "shared tree" else "dynamic", counts=[6, 5, 6])
    if case == "negative length":
        c["seq_lens"][1] = -1
    elif case == "too long":
        c["seq_lens"][1] = c["block_table"].shape[1] * 16 - 4
    elif case == "count":
        c["n_nodes"][1] = 7
    elif case == "negative count":
        c["n_nodes"][1] = -2
    elif case == "root":
        c["parent"][1, 0] = 0
    elif case == "parent":
        c["parent"][1, 4] = 4
    elif case == "block":
        c["block_table"][1, 2] = c["k_cache"].shape[0]
    elif case == "negative block":
        c["block_table"][1, 2] = -5
    else:
        c["parent"][3] = 5
    run(c, error)


def test_another_stream_and_a_graph():
    c = make(3, 5, 8, 2, 128, 16, [300, 50, 0], seed=12)
    d = on_gpu(c)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = _svp().tree_attention(**d, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    want = _svp().tree_attention(**d)
    assert torch.equal(got["out"], want["out"])
    out = _svp().tree_attention(**d)  # buffers of the graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _svp().tree_attention(**d, out=out)
    d["q"].copy_(d["q"].flip(0))
    d["seq_lens"].copy_(torch.tensor([20, 10, 0]))
    for _ in range(2):
        out["out"].zero_()
        graph.replay()
    assert torch.equal(out["out"], _svp().tree_attention(**d)["out"])
    c["q"], c["seq_lens"] = c["q"].flip(0), torch.tensor([20, 10, 0], dtype=torch.int32)
    assert int(out["dev_error"]) == 0
    want, bound = ref.attend(*[c[x] for x in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "parent",
                                              "n_nodes", "scale")])
    # request 1's and 0's nodes now lie where their sequences were
    assert bool(((out["out"].double().cpu() - want).abs() <= bound)[:2].all())


def test_two_calls_at_once():
    """On two streams, with buffers of their own, again and again: the same bits as alone."""
    cases = [on_gpu(make(4, 5, 8, 2, 128, 16, [900, 30, 2000, 0], seed=20)),
             on_gpu(make(3, 40, 8, 2, 64, 64, [700, 50, 1500], form="dynamic", seed=21))]
    want = [_svp().tree_attention(**c)["out"] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [{} for _ in cases]
    for _ in range(20):
        for c, out, stream in zip(cases, outs, streams):
            _svp().tree_attention(**c, out=out, stream=stream)
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out["out"], w) and int(out["dev_error"]) == 0

"""adjust_logits against the definition in 64 bits: types, odd vocabularies, histories, drafts, biases, masks."""

import numpy as np
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu


def _svp():
    import speculative_decoding_verification_60_gb300 as svp

    return svp


def make(B, R, V, dtype=torch.bfloat16, L=50, form="chain", bias=6, allow=0.5, pad=0, seed=0, counts=None, whole=None):
    rng = np.random.default_rng(seed)
    x = torch.tensor(rng.normal(0, 3, (B, R, V + pad)), dtype=torch.float32).to(dtype)[:, :, :V]
    ids = lambda *s: (rng.random(s) ** 3 * V).astype(np.int32)  # noqa: E731  (low ids again and again)
    c = dict(logits=x, history=ids(B, L), history_lens=rng.integers(0, L + 1, B).astype(np.int32))
    c["history_lens"][0] = L
    c["prompt_lens"] = (c["history_lens"] * rng.random(B)).astype(np.int32)
    nodes = ids(B, R)
    if form == "chain":
        c["parent"] = None
        c["drafted"] = nodes if whole else nodes[:, 1:]
    else:
        c["parent"] = np.array([ref.random_tree(R, 6, rng) for _ in range(1 if form == "tree" else B)], np.int32)
        if form == "tree":
            c["parent"] = c["parent"][0]
        c["drafted"] = nodes
    c["n_nodes"] = None if counts is None else np.resize(counts, B).astype(np.int32)
    c["repetition"] = (rng.random(B) + 0.7).astype(np.float32)
    c["frequency"] = (rng.random(B) - 0.3).astype(np.float32)
    c["presence"] = (rng.random(B) - 0.3).astype(np.float32)
    if bias:
        c["bias_ids"] = ids(B, bias)
        c["bias_ids"][:, -1] = -1
        c["bias_ids"][:, 0] = c["bias_ids"][:, bias // 2]  # one id twice
        c["bias_values"] = rng.normal(0, 5, (B, bias)).astype(np.float32)
    if allow is not None:
        words = rng.random((B, R, (V + 31) // 32, 32)) < allow
        c["allowed"] = (words * (1 << np.arange(32))).sum(3).astype(np.uint32).view(np.int32)
    return c


def run(c, error=0, in_place=False, keep=None):
    x = c["logits"]
    B, R, V = x.shape
    d = {k: torch.as_tensor(np.ascontiguousarray(t)).cuda() for k, t in c.items() if t is not None and k != "logits"}
    x_gpu = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)
    if keep is not None:
        d.update(keep)
    out = dict(logits=x_gpu) if in_place else dict(logits=torch.full((B, R, V), 7.0, dtype=x.dtype, device="cuda"))
    got = _svp().adjust_logits(x_gpu, **d, out=out)
    assert int(got["dev_error"]) == error
    y = got["logits"].double().cpu().numpy()
    get = lambda k: c.get(k)  # noqa: E731
    drafted = get("drafted")
    if drafted is not None and drafted.shape[1] == R - 1:
        drafted = np.concatenate([np.zeros((B, 1), np.int32), drafted], 1)
    u = ref.half_step(x.dtype)
    for b in range(B):
        n = R
        if get("n_nodes") is not None and 0 <= c["n_nodes"][b] <= R:
            n = int(c["n_nodes"][b])
        tree = np.arange(-1, R - 1) if get("parent") is None else c["parent"] if c["parent"].ndim == 1 else c["parent"][b]
        for i in range(n):
            raw = x[b, i].double().numpy()
            want = ref.adjust(raw, b, i, get("history"), get("history_lens"), get("prompt_lens"), drafted, tree[:n],
                              *[get(k) for k in ("repetition", "frequency", "presence", "bias_ids", "bias_values",
                                                 "allowed")])
            inf = np.isinf(want)
            assert np.array_equal(y[b, i][inf], want[inf]), (b, i)
            # a rounding to the type, and some in 32 bits of the largest term
            terms = np.abs(raw) * 3 + np.abs(np.where(inf, 0.0, want)) + 50.0 * 3
            if get("bias_ids") is not None:
                terms = terms + np.abs(c["bias_values"][b]).sum()
            off = np.abs(y[b, i][~inf] - want[~inf])
            assert (off <= np.abs(want[~inf]) * u + 8 * 2.0**-24 * terms[~inf]).all(), (b, i, off.max())
        rest = y[b, n:]
        assert (rest == (x[b, n:].double().numpy() if in_place else 7.0)).all()
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 5, 32, 33, 1000, 1001, 8192, 8193, 20011])
def test_vocabularies(dtype, V):
    run(make(3, 4, V, dtype))


@pytest.mark.parametrize("R", [1, 2, 9, 33])
@pytest.mark.parametrize("form", ["chain", "tree", "dynamic"])
def test_drafts(R, form):
    run(make(3, R, 500, form=form, seed=R))


@pytest.mark.parametrize("L", [1, 255, 256, 257, 5000])
def test_histories(L):
    run(make(4, 3, 9000, torch.float32, L=L, seed=L))


@pytest.mark.parametrize("gone", ["history", "drafted", "bias", "allowed", "penalties", "all"])
def test_groups_that_are_not_given(gone):
    c = make(3, 4, 777)
    groups = dict(history=["history", "history_lens", "prompt_lens"], drafted=["drafted", "parent"],
                  bias=["bias_ids", "bias_values"], allowed=["allowed"],
                  penalties=["repetition", "frequency", "presence"])
    for name in groups if gone == "all" else [gone]:
        for key in groups[name]:
            c.pop(key, None)
    got = run(c)
    if gone == "all":
        assert torch.equal(got["logits"].cpu(), c["logits"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strides_and_in_place(dtype, pad):
    run(make(3, 4, 1001, dtype, pad=pad))  # rows of other alignments than the output's
    run(make(3, 4, 1001, dtype, pad=pad, seed=1), in_place=True)
    run(make(2, 3, 8200, dtype, seed=2, form="tree"), in_place=True)


@pytest.mark.parametrize("allow", [0.0, 0.003, 0.99, 1.0])
def test_masks(allow):
    c = make(3, 4, 3000, allow=allow)
    if allow == 0.0:
        assert np.isneginf(run(c)["logits"].float().cpu().numpy()).all()
    else:
        run(c)


def test_what_a_mask_hides():
    """NaN, infinities and the lowest value: hidden, they are -inf; seen, they act by the formula."""
    c = make(1, 2, 700, torch.float32, bias=0, allow=1.0)
    low = torch.finfo(torch.float32).min
    c["logits"][0, :, 100:104] = torch.tensor([float("nan"), float("inf"), -float("inf"), low])
    c["logits"][0, :, 600:604] = torch.tensor([float("nan"), float("inf"), -float("inf"), low])
    c["allowed"][0, :, 100 // 32] = 0
    for v in (600, 601, 602, 603):
        c["history"][c["history"] == v] = 0
        c["drafted"][c["drafted"] == v] = 0
    y = _svp().adjust_logits(c["logits"].cuda(), **{k: torch.as_tensor(np.ascontiguousarray(t)).cuda()
                                                    for k, t in c.items() if t is not None and k != "logits"})["logits"].cpu()
    assert torch.isneginf(y[0, :, 96:128]).all()
    assert torch.isnan(y[0, :, 600]).all() and (y[0, :, 601] == float("inf")).all()
    assert torch.isneginf(y[0, :, 602]).all() and (y[0, :, 603] == low).all()


def test_counts():
    run(make(5, 7, 600, counts=[7, 0, 3, 1, 6], form="dynamic"))
    run(make(5, 7, 600, counts=[7, 0, 3, 1, 6], form="chain", whole=True), in_place=True)


@pytest.mark.parametrize("case,error", [("history", 1), ("drafted", 1), ("bias", 1), ("lens", 8), ("negative lens", 8),
                                        ("prompt", 8), ("count", 8), ("parent", 4), ("root", 4)])
def test_faulty_data(case, error):
    c = make(3, 5, 400, form="dynamic", counts=[5, 5, 4])
    if case == "history":
        c["history"][0, 3], c["history"][0, 4] = 400, -7
    elif case == "drafted":
        c["drafted"][1, 2] = 12345
    elif case == "bias":
        c["bias_ids"][1, 2] = -2
    elif case == "lens":
        c["history_lens"][1] = 51
    elif case == "negative lens":
        c["history_lens"][1] = -1
        c["prompt_lens"][1] = 0
    elif case == "prompt":
        c["prompt_lens"][1] = -4
    elif case == "count":
        c["n_nodes"][1] = 6
    elif case == "parent":
        c["parent"][1, 3] = 3
    else:
        c["parent"][1, 0] = 2
    run(c, error)


def test_many_biases_and_a_long_chain():
    run(make(1, 300, 2000, bias=1000, L=3000, seed=4))


def test_the_largest_vocabulary():
    run(make(1, 2, 524280, L=4000, bias=300, seed=5))


def test_a_graph():
    c = make(3, 4, 5000, seed=6)
    d = {k: torch.as_tensor(t).contiguous().cuda() for k, t in c.items() if t is not None}
    out = _svp().adjust_logits(**d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _svp().adjust_logits(**d, out=out)
    d["history"].random_(0, 5000)
    d["logits"].neg_()
    graph.replay()
    assert torch.equal(out["logits"], _svp().adjust_logits(**d)["logits"])

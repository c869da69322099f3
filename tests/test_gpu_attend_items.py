"""tree_attention where a CTA has many items of two blocks of rows one after the other, some of them without a second:
against the definition in 64 bits, with the error word at 0 and the same bits every time."""

import numpy as np
import pytest
import torch

import attend_matrix
from test_gpu_attend import make, on_gpu

pytestmark = pytest.mark.gpu


def run(c):
    import speculative_decoding_verification_60_gb300 as svp

    want, bound = attend_matrix.attend(*[c[x] for x in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "parent",
                                                        "n_nodes", "scale")])
    d = on_gpu(c)
    out = dict(out=torch.full(c["q"].shape, 7.0, dtype=c["q"].dtype, device="cuda"))
    got = svp.tree_attention(**d, out=out)["out"].clone()
    assert int(out["dev_error"]) == 0
    again = svp.tree_attention(**d, out=out)["out"]
    assert int(out["dev_error"]) == 0 and torch.equal(torch.nan_to_num(again, nan=9.0), torch.nan_to_num(got, nan=9.0))
    got = got.double().cpu()
    B, N = got.shape[:2]
    live = torch.ones(B, N, dtype=torch.bool) if c["n_nodes"] is None else torch.arange(N) < c["n_nodes"][:, None]
    assert bool((got[~live] == 7.0).all())  # rows behind a request's nodes stay
    got, want, bound = got[live], want[live], bound[live]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    off = torch.nan_to_num((got - want).abs() - bound, nan=-1.0)
    assert float(off.max()) <= 0, float(off.max())
    return want


def not_finite(c, values):
    """values: {request: (node, key head, value)}."""
    page = c["k_cache"].shape[1]
    for b, (node, head, value) in values.items():
        t = int(c["seq_lens"][b]) + node
        c["v_cache"][int(c["block_table"][b, t // page]), t % page, head, 3] = value


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_tree_of_forty_nodes(dtype, dim):
    """Two and a half blocks of rows: the CTAs of the second share never have a second block."""
    lens = np.random.default_rng(0).integers(0, 300, 64)
    run(make(64, 40, 64, 8, dim, 16, lens, dtype, form="tree", seed=1))


@pytest.mark.parametrize("dim", [64, 96, 128])
def test_small_trees_in_a_buffer_of_sixty(dim):
    """Counts within one block of two, 128 requests: no item has a second block."""
    rng = np.random.default_rng(2)
    run(make(128, 60, 64, 8, dim, 16, rng.integers(0, 90, 128), form="dynamic", counts=rng.integers(1, 17, 128), seed=2))


@pytest.mark.parametrize("counts", ["one to sixty", "about a block", "about two blocks", "some none"])
def test_counts_about_the_blocks_ends(counts):
    rng = np.random.default_rng(3)
    n = dict([("one to sixty", rng.integers(1, 61, 100)), ("about a block", rng.integers(15, 19, 100)),
              ("about two blocks", rng.integers(31, 35, 100)), ("some none", rng.integers(0, 3, 100) * 16)])[counts]
    run(make(100, 60, 64, 8, 64, 32, rng.integers(0, 260, 100), form="dynamic", counts=n, seed=3))


@pytest.mark.parametrize("N", [65, 80])
def test_a_group_of_four(N):
    rng = np.random.default_rng(4)
    run(make(64, N, 32, 8, 64, 16, rng.integers(0, 200, 64), form="tree", seed=4))


def test_one_block_too_many_in_every_request():
    lens = np.random.default_rng(5).integers(0, 95, 128)
    run(make(128, 33, 64, 8, 128, 16, lens, form="chain", seed=5))


@pytest.mark.parametrize("N,counts", [(17, 16), (33, None), (20, None), (3, None)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_request(N, counts, value):
    """Short requests, one of them with a value that is not finite in one node: its rows that see the node, of that
    key head, are NaN, and no others."""
    B = 120
    lens = np.random.default_rng(6).integers(0, 128 - N, B)
    c = make(B, N, 64, 8, 64, 16, lens, counts=None if counts is None else [counts], seed=6)
    not_finite(c, {50: (1, 5, value)})
    want = torch.isnan(run(c))
    assert int(want.all(2).sum()) == int(want.any(2).sum()) == ((N if counts is None else counts) - 1) * 8


def test_what_is_not_finite_in_items_one_after_the_other():
    rng = np.random.default_rng(7)
    B = 120
    c = make(B, 33, 64, 8, 64, 16, rng.integers(0, 95, B), form="dynamic", counts=rng.integers(2, 34, B), seed=7)
    not_finite(c, {b: (int(c["n_nodes"][b]) - 1 - b % 2, b % 8, (float("nan"), float("inf"), -float("inf"))[b % 3])
                   for b in range(B) if b % 5 < 3})
    run(c)

"""Pins of the 64-bit reference of the calls over vocabulary rows and cache
blocks, and the refusals of those calls (no GPU needed)."""

import ctypes

import numpy as np
import pytest

import vocab_reference as ref


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_60_gb300 import build

    build.build()
    import speculative_decoding_verification_60_gb300 as svp

    return svp.load()


def test_reference_logprobs_by_hand():
    x = np.log(np.array([[0.5, 0.125, 0.25, 0.125]], np.float32))
    out, err = ref.token_logprobs(x, [3], 1.0, 4)
    assert err == 0 and out["rank"][0] == 4 and list(out["top_ids"][0]) == [0, 2, 1, 3]
    assert np.isclose(out["logprob"][0], np.log(0.125)) and np.isclose(out["entropy"][0], 1.75 * np.log(2))


@pytest.mark.parametrize("bucket", [False, True])
@pytest.mark.parametrize("T", [0.6, 1.0, 2.0])
def test_reference_gradient_against_differences(bucket, T):
    rng = np.random.default_rng(3)
    V, K = 23, 5
    s = rng.normal(size=V) * 2
    teacher = ref.log_softmax(rng.normal(size=V) * 2, 1.0)
    ids = ref.order(teacher)[:K].copy()
    l = teacher[ids]
    ids[3] = -1
    loss, g, _, err = ref.distill_row(s, ids, l, T, bucket)
    assert err == 0 and loss > 0
    h = 1e-6
    for v in range(V):
        e = np.zeros(V)
        e[v] = h
        d = (ref.distill_row(s + e, ids, l, T, bucket)[0] - ref.distill_row(s - e, ids, l, T, bucket)[0]) / (2 * h)
        assert abs(d - g[v]) < 1e-8  # h^2 plus 2^-53 |loss| / h


def test_reference_loss_is_zero_at_the_teacher():
    rng = np.random.default_rng(4)
    s = rng.normal(size=50)
    lp = ref.log_softmax(s, 1.0)
    ids = ref.order(s)[:7]
    loss, g, _, _ = ref.distill_row(s, ids, lp[ids], 1.0, True)
    assert abs(loss) < 1e-14 and np.abs(g).max() < 1e-15


def test_reference_blocks_by_hand():
    table = np.full((3, 4), -1, np.int32)
    table[0, 0], table[1, :2], table[2, 0] = 7, [8, 9], 5
    free = np.array([20, 21, 22, 23], np.int32)
    out, err = ref.advance_blocks([3, 7, 2], [0, -1, 1], [5, 1, 1], 4, table, [1, 2, 1], free, 3, 8)
    # request 0: length 4 and five more, so blocks 1 and 2, from the end of the three entries in use;
    # request 1: position 7 is in the block it has; request 2: position 4 opens its second block
    assert err == 0 and out["table"].tolist() == [[7, 22, 21, -1], [8, 9, -1, -1], [5, 20, -1, -1]]
    assert out["slots"].tolist() == [88, 89, 90, 91, 84, 39, 80, -1]
    assert out["positions"].tolist() == [4, 5, 6, 7, 8, 7, 4, 0]
    assert out["cu_tokens"].tolist() == [0, 5, 6, 7] and out["free_count"] == 0
    assert out["seq_lens"].tolist() == [4, 7, 4] and out["held"].tolist() == [3, 2, 2]
    # with two entries free, request 0 takes both and request 2 is left out
    out, err = ref.advance_blocks([3, 7, 2], [0, -1, 1], [5, 1, 1], 4, table, [1, 2, 1], free, 2, 8)
    assert err == ref.DEVERR_CAPACITY and out["slots"].tolist() == [84, 85, 86, 87, 80, 39, -1, -1]
    assert out["held"].tolist() == [3, 2, 1] and out["free_count"] == 0


def _status(lib, name, good, **change):
    """Status of a call with one argument of a good set changed."""
    args = dict(good)
    args.update(change)
    return getattr(lib, name)(*args.values())


def test_token_logprobs_refusals(lib):
    d = ctypes.c_void_p(16)
    good = dict(logits=d, dtype=0, R=2, V=64, stride=64, tokens=d, T=1.0, K=4, logprob=d, rank=d, entropy=d, ids=d,
                lps=d, err=d, stream=None)
    bad = lambda **k: _status(lib, "spec_token_logprobs", good, **k)  # noqa: E731
    for change in (dict(logits=None), dict(dtype=5), dict(R=-1), dict(V=0), dict(stride=63), dict(T=0.0),
                   dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(K=-1), dict(K=65),
                   dict(logprob=None), dict(ids=None), dict(lps=None)):
        assert bad(**change) == 1, change
    assert bad(V=1000, stride=1000, K=129) == 2
    assert bad(V=524281, stride=524281) == 2
    assert bad(R=0, err=None) == 0


def test_distill_refusals(lib):
    d, e = ctypes.c_void_p(16), ctypes.c_void_p(32)
    good = dict(student=d, dtype=0, R=2, V=64, stride=64, ids=d, lp=d, K=4, w=None, T=1.0, tail=1, loss=d, stats=None,
                grad=e, grad_stride=64, err=None, stream=None)
    bad = lambda **k: _status(lib, "spec_distill_topk", good, **k)  # noqa: E731
    for change in (dict(student=None), dict(dtype=2), dict(R=-1), dict(V=0), dict(stride=10), dict(ids=None),
                   dict(lp=None), dict(K=0), dict(T=0.0), dict(tail=2), dict(loss=None), dict(grad_stride=63),
                   dict(grad=d, grad_stride=65)):
        assert bad(**change) == 1, change
    assert bad(K=129) == 2 and bad(V=524281, stride=524281, grad=None) == 2 and bad(R=0) == 0
    good = dict(student=d, dtype=0, R=2, V=64, stride=64, ids=d, lp=d, K=4, stats=d, gl=None, T=1.0, grad=e,
                grad_stride=64, stream=None)
    bad = lambda **k: _status(lib, "spec_distill_topk_backward", good, **k)  # noqa: E731
    for change in (dict(student=None), dict(stats=None), dict(grad=None), dict(ids=None), dict(lp=None), dict(K=0),
                   dict(T=float("nan")), dict(stride=63), dict(grad_stride=63)):
        assert bad(**change) == 1, change
    assert bad(K=129) == 2 and bad(R=0) == 0


def test_advance_blocks_refusals(lib):
    d, e = ctypes.c_void_p(16), ctypes.c_void_p(32)
    good = dict(lens=d, acc=None, new=d, B=2, page=16, table=d, M=4, stride=4, held=d, free=d, cap=8, count=d,
                olens=e, oheld=e, ocount=e, cu=e, slots=e, pos=None, T=16, err=None, stream=None)
    bad = lambda **k: _status(lib, "spec_advance_blocks", good, **k)  # noqa: E731
    for change in (dict(lens=None), dict(new=None), dict(B=0), dict(page=0), dict(table=None), dict(M=0),
                   dict(stride=3), dict(held=None), dict(free=None), dict(cap=-1), dict(count=None), dict(olens=None),
                   dict(oheld=None), dict(ocount=None), dict(cu=None), dict(slots=None), dict(T=-1),
                   dict(olens=d), dict(oheld=d), dict(ocount=d)):
        assert bad(**change) == 1, change
    assert bad(B=16385) == 2
    assert bad(B=16384, M=200000, stride=200000) == 2


def test_bindings_refuse_what_the_calls_cannot_take(lib):
    import torch

    import speculative_decoding_verification_60_gb300 as svp

    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        svp.token_logprobs(x)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        svp.token_logprobs(x.half())
    with pytest.raises(ValueError, match="CUDA"):
        svp.distill_topk(x, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4))
    with pytest.raises(TypeError, match="int32"):
        svp.advance_blocks(*[torch.zeros(2, dtype=torch.int32)] * 2, torch.zeros(2, 4), *[None] * 3, 16, 8)

"""spec_token_logprobs against the 64-bit reference: identifiers and ranks
equal, log probabilities and entropies within the bound of 32-bit sums."""

import numpy as np
import pytest
import torch

import synth
import vocab_reference as ref

pytestmark = pytest.mark.gpu
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _svp():
    import speculative_decoding_verification_60_gb300 as svp

    return svp


def _logits(R, V, dtype, seed):
    if dtype == "bf16":
        return synth.zipf_logits(R, V, seed)
    return synth.zipf_logits(R, V, seed).float() + synth.gaussian((R, V), 0.01, seed + 1)


def _place(x, pad=0, offset=0):
    """x on the GPU as rows of a wider buffer that starts `offset` elements in."""
    R, V = x.shape
    buf = torch.full((offset + R * (V + pad),), 77.0, dtype=x.dtype, device="cuda")
    view = buf[offset:].view(R, V + pad)[:, :V]
    view.copy_(x)
    return view


def _check(x, tokens, T, K, placed=None, rows=None):
    dev = placed if placed is not None else x.cuda()
    tok = None if tokens is None else torch.as_tensor(tokens, dtype=torch.int32).cuda()
    got = _svp().token_logprobs(dev, tok, T, K)
    got = {k: v.cpu().numpy() for k, v in got.items()}
    rows = list(range(x.shape[0])) if rows is None else rows
    want, err = ref.token_logprobs(x[rows].float().numpy(), None if tokens is None else np.asarray(tokens)[rows], T, K)
    assert len(rows) < x.shape[0] or got["dev_error"][0] == err
    assert np.array_equal(got["top_ids"][rows], want["top_ids"])
    assert np.array_equal(got["rank"][rows], want["rank"])
    bound = ref.sum_bound(x.shape[1])
    for key in ("logprob", "top_logprobs", "entropy"):
        g, w = got[key][rows].astype(np.float64), want[key]
        fine = np.isfinite(w)
        assert np.array_equal(g[~fine], w[~fine]), key
        # (x - m) / T, its difference with ln Z and the result are rounded: 4 units of the value
        tol = bound * (1 + (np.abs(w) if key == "entropy" else 0)) + 4 * ref.EPS * np.abs(w)
        assert (np.abs(g - w)[fine] <= tol[fine]).all(), (key, np.abs(g - w)[fine].max())
    return got


def _tokens(x, seed):
    rng = np.random.default_rng(seed)
    t = rng.integers(0, x.shape[1], x.shape[0])
    best = x.float().argmax(1).numpy()
    return np.where(rng.random(x.shape[0]) < 0.5, t, best).astype(np.int32)


@pytest.mark.parametrize("V,K", [(1, 1), (2, 2), (7, 3), (31, 31), (32, 8), (33, 20), (255, 128), (256, 1), (1001, 64),
                                 (4097, 128), (16384, 20), (16392, 5), (50021, 20), (128256, 20), (129280, 128),
                                 (262144, 33), (524280, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_vocabularies(V, K, dtype):
    R = 5 if V > 200000 else 9
    x = _logits(R, V, dtype, seed=V + K)
    _check(x, _tokens(x, V), 0.8, K)


@pytest.mark.parametrize("R", [1, 2, 3, 19, 38, 40, 77, 153, 200, 700, 1300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_counts(R, dtype):
    # every way of sharing rows among the SMs, from one row split over several to many rows each
    x = _logits(R, 20000, dtype, seed=R)
    rows = sorted(np.random.default_rng(R).choice(R, min(R, 24), replace=False).tolist())
    _check(x, _tokens(x, R), 1.0, 20, rows=rows)


@pytest.mark.parametrize("T", [0.05, 0.7, 1.0, 5.0])
def test_temperatures(T):
    x = _logits(6, 8192, "bf16", seed=5)
    _check(x, _tokens(x, 5), T, 10)


@pytest.mark.parametrize("V,pad,offset", [(1000, 0, 1), (1001, 0, 0), (1001, 7, 3), (4096, 5, 2), (50000, 24, 8),
                                          (9, 1, 5), (128256, 3, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_alignment(V, pad, offset, dtype):
    x = _logits(7, V, dtype, seed=V)
    _check(x, _tokens(x, V), 1.0, min(V, 20), placed=_place(x, pad, offset))


def test_leading_shape_of_a_verification():
    svp = _svp()
    x = _logits(12, 2000, "bf16", seed=8)
    tok = torch.as_tensor(_tokens(x, 8)).view(4, 3).cuda()
    tok[1, 2] = -1
    got = svp.token_logprobs(x.cuda().view(4, 3, 2000), tok, 1.0, 5)
    flat = svp.token_logprobs(x.cuda(), tok.view(-1), 1.0, 5)
    assert got["top_ids"].shape == (4, 3, 5) and got["logprob"].shape == (4, 3)
    for k in ("logprob", "rank", "entropy", "top_ids", "top_logprobs"):
        assert torch.equal(got[k].flatten(), flat[k].flatten())


def test_skipped_rows_are_not_read():
    x = _logits(6, 3000, "bf16", seed=9)
    tok = _tokens(x, 9)
    tok[[1, 4]] = -1
    x[1] = float("nan")
    x[4] = float("inf")
    got = _check(x, tok, 1.0, 4)
    assert got["dev_error"][0] == 0 and got["rank"][1] == -1 and got["logprob"][4] == 0


@pytest.mark.parametrize("V", [40, 3000, 50021, 128256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks(V, dtype):
    K = min(V, 64)
    x = _logits(9, V, dtype, seed=V)
    low = torch.finfo(DTYPE[dtype]).min
    rng = np.random.default_rng(V)
    keep = lambda n: torch.as_tensor(rng.choice(V, n, replace=False))  # noqa: E731
    for r, n in ((0, 1), (1, 5), (2, min(V, 100)), (3, V // 2)):  # fewer finite entries than alternatives, and more
        y = torch.full((V,), -float("inf"), dtype=x.dtype)
        k = keep(n)
        y[k] = x[r][k]
        x[r] = y
    x[4] = low  # every entry the type's lowest value: uniform
    y = torch.full((V,), low, dtype=x.dtype)
    k = keep(3)
    y[k] = x[5][k]
    x[5] = y
    x[6, : V // 2] = -float("inf")
    x[6, V // 2:] = low
    x[7] = 0.0
    x[7, ::2] = -0.0  # equal to +0: the order is by index
    tok = x.float().argmax(1).numpy().astype(np.int32)
    tok[3] = int(torch.nonzero(x[3] == -float("inf"))[0]) if V > 2 else 0  # a token that is ruled out
    got = _check(x, tok, 1.0, K)
    assert got["dev_error"][0] == 0
    _check(x, tok, 0.25, K)


@pytest.mark.parametrize("V", [300, 20000, 128256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 20, 128])
def test_ties_and_sorted_rows(V, dtype, K):
    ramp = torch.linspace(-9, 9, V)
    x = torch.stack([torch.full((V,), 1.5), ramp, ramp.flip(0), torch.round(ramp), torch.round(ramp).flip(0),
                     (torch.arange(V) % 7 == 3).float(), (torch.arange(V) % 1009 == 5).float(),
                     (torch.arange(V) == V - 1).float()]).to(DTYPE[dtype])
    _check(x, _tokens(x, V), 1.0, K)


def test_the_rank_of_a_token_that_is_ruled_out():
    """Every place in the row, its unaligned ends too, among -inf entries."""
    for V, offset in ((1003, 0), (1003, 3), (2500, 5)):
        x = torch.full((12, V), -float("inf"), dtype=torch.bfloat16)
        x[:, ::3] = synth.gaussian((12, len(range(0, V, 3))), 1.0, V).to(torch.bfloat16)
        tok = np.array([1, 2, 4, 7, 8, 256, 259, 770, V - 5, V - 3, V - 2, V - 1], np.int32)
        _check(x, tok, 1.0, 3, placed=_place(x, 0, offset))


def test_large_magnitudes():
    x = synth.gaussian((4, 5000), 1.0, 3)
    x[0] *= 1e4
    x[1] = x[1] * 1e-4 + 3e4
    x[2, 17] = 3e38
    x[3] = -x[3].abs() * 1e38
    _check(x, _tokens(x, 3), 1.0, 16)


def test_refused_rows_and_their_neighbours():
    V = 3001
    x = _logits(8, V, "bf16", seed=10)
    tok = _tokens(x, 10)
    x[1, 17] = float("nan")
    x[2, V - 1] = float("inf")
    x[3] = -float("inf")
    tok[5], tok[6] = V, -2
    got = _check(x, tok, 1.0, 6)
    assert got["dev_error"][0] == 3
    # the error word is of the last call alone
    assert _check(x[7:], tok[7:], 1.0, 6)["dev_error"][0] == 0
    # without tokens the same rows are refused for their values only
    assert _check(x, None, 1.0, 6)["dev_error"][0] == 2


@pytest.mark.parametrize("V", [20, 700, 30000, 100000, 262144])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_full_of_what_is_refused(V, dtype, bad):
    """All of the row, half of it, every 50th element, one run: no answer, and an end to the search for one."""
    x = _logits(6, V, dtype, seed=V)
    x[1] = bad
    x[2, V // 2:] = bad
    x[3, ::50] = bad
    x[4, : V // 3] = -float("inf")
    x[4, V // 3: V // 2] = bad
    for K in (0, 7, min(V, 128)):
        assert _check(x, _tokens(x, V), 1.0, K)["dev_error"][0] == 2


def test_no_tokens_no_alternatives_no_rows():
    svp = _svp()
    x = _logits(5, 700, "f32", seed=11)
    _check(x, None, 1.0, 12)
    _check(x, _tokens(x, 1), 1.0, 0)
    got = svp.token_logprobs(x[:0].cuda(), torch.empty(0, dtype=torch.int32, device="cuda"), 1.0, 4)
    assert got["logprob"].shape == (0,) and got["top_ids"].shape == (0, 4) and int(got["dev_error"]) == 0


def test_offsets_past_32_bits():
    V, stride = 1000, 2**31 + 8
    buf = torch.empty(stride + V, dtype=torch.bfloat16, device="cuda")
    rows = buf.as_strided((2, V), (stride, 1))
    x = _logits(2, V, "bf16", seed=12)
    rows.copy_(x)
    _check(x, _tokens(x, 12), 1.0, 20, placed=rows)


def test_same_bits_every_time_and_on_another_stream():
    svp = _svp()
    x = _logits(40, 128256, "bf16", seed=13).cuda()
    tok = torch.as_tensor(_tokens(x.cpu(), 13)).cuda()
    first = svp.token_logprobs(x, tok, 0.9, 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = svp.token_logprobs(x, tok, 0.9, 20, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    one = svp.token_logprobs(x[7:8], tok[7:8], 0.9, 20)
    for k in first:
        assert torch.equal(first[k], again[k]), k
    for k in ("rank", "top_ids"):
        assert torch.equal(first[k][7:8], one[k]), k


def test_captured_in_a_graph():
    svp = _svp()
    x = _logits(8, 5000, "bf16", seed=14).cuda()
    tok = torch.as_tensor(_tokens(x.cpu(), 14)).cuda()
    out = svp.token_logprobs(x, tok, 1.0, 5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svp.token_logprobs(x, tok, 1.0, 5, out=out)
    y = _logits(8, 5000, "bf16", seed=15)
    x.copy_(y)
    g.replay()
    want = svp.token_logprobs(x, tok, 1.0, 5)
    for k in want:
        assert torch.equal(out[k], want[k]), k

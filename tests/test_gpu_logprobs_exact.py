"""How exact log probabilities and entropies are: rows where one token holds
nearly all of the mass, where it rises through the row, unaligned and short
rows, every temperature; against 64 bits, to the roundings of the kernel's sums."""

import numpy as np
import pytest
import torch

import vocab_reference as ref
from test_gpu_logprobs import DTYPE, _place

pytestmark = pytest.mark.gpu
EPS = ref.EPS


def _exact(x, T, itemsize):
    """ln z against the maximum, the entropy, and the bounds of both; x in 64 bits.

    With u = (m - x) / T: a weight 2^t carries 4 units of 2^-24 of ex2, and u + 1 of the rounding of t (twice that
    where x - m is rounded, too).  Summed by two adds in a vector, six in a tile, the tiles of a warp, six over its
    lanes, nine over the warps; one more weight (5 units) brings the sum to the maximum's place.  A maximum that has
    none of an eighth of its weight beside it is counted.  ln(1 + rest) is off by what the rest is, times
    rest / (1 + rest), and by two roundings; where the rest is an eighth or more, by the maximum's weight (5) and the
    roundings of the parts (8).  The entropy adds the mean of u, whose terms are chained through the tiles of a warp
    (24 each) and whose weights go with the rounded c: one unit of 1 + u."""
    m = x.max()
    with np.errstate(all="ignore"):
        u = (m - x) / T
    u = u[np.isfinite(u)]
    w = np.exp(-u)
    rest_w, rest_u = w[u > 0], u[u > 0]
    n = int((u == 0).sum())
    rest = rest_w.sum()
    ln_z = np.log1p(rest + (n - 1))
    if n == 1:
        ln_z = np.log1p(rest)
    z = n + rest
    mean = (w * u).sum() / z
    tiles = len(x) * itemsize / 16 / 32 / 48 + 1
    far = (rest_w * rest_u).sum() / rest if rest > 0 else 0.0
    far2 = (rest_w * rest_u ** 2).sum() / (rest_w * rest_u).sum() if rest > 0 and (rest_w * rest_u).sum() > 0 else 0.0
    rho = EPS * (34 + tiles + 2 * far)
    large = n > 1 or rest > 0.12
    gone = len(x) * 2.0 ** -126  # weights that 32 bits flush
    off = rest / z * rho + (13 * EPS if large else 2 * EPS * ln_z) + gone
    off_h = off + mean * EPS * (40 + 24 * tiles + 3 * far2) + (rho + 13 * EPS if large else 0) + gone * 90
    return m, ln_z, ln_z + mean, off, off_h + 4 * EPS * (ln_z + mean)


def _check(x, T, tokens, placed=None):
    import speculative_decoding_verification_60_gb300 as svp

    T = float(np.float32(T))
    got = svp.token_logprobs(x.cuda() if placed is None else placed, torch.as_tensor(tokens, dtype=torch.int32).cuda(), T,
                             min(5, x.shape[1]))
    assert int(got["dev_error"]) == 0
    got = {k: v.double().cpu().numpy() for k, v in got.items()}
    rows = x.double().numpy()
    for r, row in enumerate(rows):
        m, ln_z, h, off, off_h = _exact(row, T, x.element_size())
        best = np.sort(row)[::-1][: got["top_logprobs"].shape[1]]
        for value, logit in [(got["logprob"][r], row[tokens[r]]), *zip(got["top_logprobs"][r], best)]:
            want = (logit - m) / T - ln_z
            if want < -np.finfo(np.float32).max:
                assert value == -np.inf
            else:
                assert abs(value - want) <= off + 4 * EPS * abs(want), (r, value, want, off)
        assert abs(got["entropy"][r] - h) <= off_h, (r, got["entropy"][r], h, off_h)


def _confident(V, dtype, T, seed):
    """One token 0 to 60 nats (of x / T) above the sum of all others, at several places of the row."""
    g = torch.Generator().manual_seed(seed)
    gaps = [-2.0, 0.0, 0.7, 2.0, 5.0, 9.0, 14.0, 20.0, 35.0, 60.0]
    x = torch.randn(len(gaps), V, generator=g, dtype=torch.float64)
    at = torch.randint(0, V, (len(gaps),), generator=g)
    at[2], at[5] = 0, V - 1
    for r, gap in enumerate(gaps):
        x[r, at[r]] = -float("inf")
        rest = torch.logsumexp(x[r] / T, 0) * T if V > 1 else torch.tensor(0.0)
        x[r, at[r]] = float(rest) + gap * T
    return x.to(DTYPE[dtype]), at.numpy().astype(np.int32)


@pytest.mark.parametrize("V", [1, 2, 9, 33, 300, 1001, 20000, 128256, 524280])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.3, 0.5, 1.0, 1.3])
def test_one_token_holds_nearly_all(V, dtype, T):
    x, at = _confident(V, dtype, T, seed=V)
    _check(x, T, at)


@pytest.mark.parametrize("V,offset,pad", [(1001, 3, 0), (7, 1, 2), (40009, 5, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_confident_rows_off_16_bytes(V, offset, pad, dtype):
    x, at = _confident(V, dtype, 0.7, seed=V)
    _check(x, 0.7, at, placed=_place(x, pad, offset))


@pytest.mark.parametrize("V", [128256, 50021])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_confident_rows_by_one_cta_each(V, dtype):
    x, at = _confident(V, dtype, 1.0, seed=V)
    g = torch.Generator().manual_seed(1)
    more = (torch.randn(80, V, generator=g) * 3).to(x.dtype)
    more[:10] = x
    _check(more, 1.0, np.concatenate([at, np.zeros(70, np.int32)]))


@pytest.mark.parametrize("V", [3000, 131072, 524280])
@pytest.mark.parametrize("T", [0.02, 0.7, 1.3, 30.0])
def test_rows_whose_maximum_rises(V, T):
    """Through the whole row, steeply and by a hair, and in two steps; several equal maxima."""
    up = torch.linspace(0, 1, V, dtype=torch.float64)
    x = torch.stack([up * 20, up * 1e-2 + 3, up * 1e-5, (up > 0.4) + 5.0 * (up > 0.8), -up * 20, torch.round(up * 40)])
    for kind in (torch.bfloat16, torch.float32):
        _check(x.to(kind), T, np.array([V - 1, 0, V // 2, V - 1, 0, V - 1]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,T", [(1e4, 1.0), (3.0, 1e-3), (3.0, 2.0 ** -126), (1e30, 1e29), (1.0, 1e30)])
def test_places_past_the_ordinary_range(scale, T, dtype):
    g = torch.Generator().manual_seed(9)
    x = (torch.randn(6, 5000, generator=g) * scale).to(DTYPE[dtype])
    x[2, :2000] = torch.finfo(x.dtype).min
    x[3, 1000:] = -float("inf")
    _check(x, T, x.float().argmax(1).numpy())

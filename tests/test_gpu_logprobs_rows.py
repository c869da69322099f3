"""spec_token_logprobs by every number of CTAs a row (8, 4, 2 and 1, by the
number of rows), with the alternatives' bound from the maxima of more than 256
groups as well as from vectors."""

import numpy as np
import pytest
import torch

from test_gpu_logprobs import DTYPE, _check, _tokens

pytestmark = pytest.mark.gpu


def _logits(R, V, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(R, V, generator=g, device="cuda") * 2).to(DTYPE[dtype])


@pytest.mark.parametrize("R", [5, 30, 31, 60, 61, 76, 77, 90, 200, 700])
@pytest.mark.parametrize("V,dtype", [(128256, "bf16"), (50021, "f32"), (128255, "bf16")])
def test_rows_and_the_ctas_that_share_them(R, V, dtype):
    x = _logits(R, V, dtype, seed=R)
    rows = sorted(np.random.default_rng(R).choice(R, min(R, 12), replace=False).tolist())
    host = x[rows].cpu()
    tokens = np.random.default_rng(R + 1).integers(0, V, R).astype(np.int32)
    tokens[rows] = _tokens(host, R)

    class Rows:  # of which only `rows` are looked at
        shape = x.shape

        def __getitem__(self, at):
            assert at == rows
            return host

    _check(Rows(), tokens, 0.9, 20, placed=x, rows=rows)


@pytest.mark.parametrize("V,dtype", [(128256, "bf16"), (50021, "f32"), (50023, "f32")])
@pytest.mark.parametrize("K", [1, 20, 128])
def test_masks_ties_and_sorted_rows_by_one_cta_each(V, dtype, K):
    """The rows of test_masks and test_ties_and_sorted_rows among 90."""
    kind = DTYPE[dtype]
    low, ninf = torch.finfo(kind).min, -float("inf")
    ramp = torch.linspace(-9, 9, V)
    some = _logits(8, V, dtype, seed=V).cpu()
    rng = np.random.default_rng(V)
    rows = [torch.full((V,), 1.5), ramp, ramp.flip(0), torch.round(ramp), torch.round(ramp).flip(0),
            (torch.arange(V) % 7 == 3).float(), (torch.arange(V) % 1009 == 5).float(), (torch.arange(V) == V - 1).float()]
    for n, fill in ((1, ninf), (5, ninf), (100, ninf), (V // 2, ninf), (3, low), (0, low)):
        y = torch.full((V,), fill, dtype=kind)
        keep = torch.as_tensor(rng.choice(V, n, replace=False))
        y[keep] = some[len(rows) % 8][keep]
        rows.append(y)
    half = torch.full((V,), low, dtype=kind)
    half[: V // 2] = ninf
    signs = torch.zeros(V)
    signs[::2] = -0.0
    rows += [half, signs]
    x = torch.stack([y.to(kind) for y in rows])
    tokens = _tokens(x, V)
    tokens[11] = int(torch.nonzero(x[11] == ninf)[0])
    many = torch.cat([x, _logits(90 - len(rows), V, dtype, seed=K).cpu()])
    got = _check(many, np.concatenate([tokens, np.zeros(90 - len(rows), np.int32)]), 1.0, K)
    assert got["dev_error"][0] == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_refused_rows_by_one_cta_each(bad):
    V = 100000
    x = _logits(84, V, "bf16", seed=3).cpu()
    x[1] = bad
    x[2, V // 2:] = bad
    x[3, ::50] = bad
    x[4, V - 1] = bad
    x[5] = -float("inf")
    assert _check(x, _tokens(x, V), 1.0, 20)["dev_error"][0] == 2

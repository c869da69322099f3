"""adjust_logits where its parameters are no ordinary numbers: repetitions whose inverse leaves the range of 32 bits, zero,
negative, infinite and NaN ones, frequencies and presences likewise; counted tokens alone are penalised.  Against the
formula in 64 bits, with histories that are counted first and ones that are not."""

import numpy as np
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
# (repetition, frequency, presence)
PARAMETERS = [(0.0, 0.3, 0.2), (2.0**-110, 0.3, -0.2), (2.0**110, -0.3, 0.2), (-1.3, 0.0, 0.5), (-(2.0**105), 0.1, 0.0),
              (INF, 0.3, 0.2), (-INF, 0.0, 0.0), (NAN, 0.5, 0.1), (1.0, NAN, 0.0), (1.0, 0.0, NAN), (1.2, INF, 0.0),
              (1.2, -INF, 0.3), (0.8, 0.4, INF), (0.8, INF, -INF), (1.0, 0.0, -INF), (2.0**-99, 0.0, 0.0)]


def formula(x, told, said, path, r, f, p, bias):
    """A row in 64 bits: tokens of the history [V], of its output and of the path (counts)."""
    with np.errstate(all="ignore"):
        seen, c = told + path > 0, said + path
        y = np.where(seen, np.where(x > 0, x / r, x * r), x)
        y = np.where(c > 0, y - (f * c + p), y)
        return y + bias


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L", [20, 400])  # 1000 / 16 lies between: counted after the rows' stream, and before it
@pytest.mark.parametrize("extra", [False, True])
def test_parameters(dtype, L, extra):
    import speculative_decoding_verification_60_gb300 as svp

    rng = np.random.default_rng(L)
    B, R, V, K = len(PARAMETERS), 4, 1000, 3
    x = torch.tensor(rng.normal(0, 3, (B, R, V)), dtype=torch.float32).to(dtype)
    x[:, :, 7] = 0.0
    history = rng.integers(0, V, (B, L)).astype(np.int32)
    history[:, 0], history[:, -1] = 7, 11
    lens, prompt = np.full(B, L, np.int32), np.full(B, L // 2, np.int32)
    r, f, p = [np.array(c, np.float32) for c in zip(*PARAMETERS)]
    d = dict(history=history, history_lens=lens, prompt_lens=prompt, repetition=r, frequency=f, presence=p)
    drafted = rng.integers(0, V, (B, R)).astype(np.int32)
    drafted[:, 2] = history[:, 1]
    parent = [-1, 0, 1, 0]
    bias_ids, bias_values = rng.integers(0, V, (B, K)).astype(np.int32), rng.normal(0, 2, (B, K)).astype(np.float32)
    bias_ids[:, 0], bias_ids[:, 1] = drafted[:, 1], history[:, 3]
    if extra:
        d.update(drafted=drafted, parent=np.array(parent, np.int32), bias_ids=bias_ids, bias_values=bias_values)
    got = svp.adjust_logits(x.cuda(), **{k: torch.as_tensor(v).cuda() for k, v in d.items()})
    assert int(got["dev_error"]) == 0
    y = got["logits"].double().cpu().numpy()
    u = ref.half_step(dtype)
    for b in range(B):
        told = np.bincount(history[b], minlength=V)
        said = np.bincount(history[b, L // 2:], minlength=V)
        bias = np.zeros(V)
        if extra:
            np.add.at(bias, bias_ids[b], bias_values[b].astype(np.float64))
        for i in range(R):
            path = np.zeros(V)
            if extra:
                np.add.at(path, [drafted[b, j] for j in ref.path(parent, i)[1:]], 1)
            raw = x[b, i].double().numpy()
            want = formula(raw, told, said, path, float(r[b]), float(f[b]), float(p[b]), bias)
            assert np.array_equal(np.isnan(y[b, i]), np.isnan(want)), (b, i)
            inf = np.isinf(want)
            assert np.array_equal(y[b, i][inf], want[inf]), (b, i)
            ok = np.isfinite(want)
            c = said + path
            with np.errstate(all="ignore"):
                terms = np.abs(want) + np.where(c > 0, np.abs(f[b].astype(np.float64)) * c + abs(float(p[b])), 0.0) + np.abs(bias)
                terms = terms + np.where(told + path > 0, np.where(raw > 0, np.abs(raw / r[b]), np.abs(raw * r[b])), np.abs(raw))
            # rounded to the type; in 32 bits two roundings of the scaled logit, one of the penalty, of each difference
            # and of the biases' sum
            off = np.abs(y[b, i][ok] - want[ok])
            assert (off <= np.abs(want[ok]) * u + 6 * 2.0**-24 * terms[ok]).all(), (b, i, off.max())

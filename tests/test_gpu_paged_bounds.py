"""How far results of the calls over a paged cache and the logits may be off, as the header states it."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [4096, 200])  # counted before the rows' stream, and after it
def test_repetitions(L):
    """x / repetition as a product with 1 / repetition: two roundings, so 2^-23 of it and a little."""
    import speculative_decoding_verification_60_gb300 as svp

    rng = np.random.default_rng(L)
    B, V = 40, 4096
    r = np.exp2(rng.uniform(-1, 1, B)).astype(np.float32)
    r[0], r[1], r[2] = 1.999976, 2.0**99, 2.0**-99
    x = np.abs(rng.normal(0, 3, (B, 1, V))).astype(np.float32) + np.float32(2.0**-10)
    x[0] = np.exp2(rng.uniform(0, 1, V)).astype(np.float32)
    x[0, 0, 0] = 1.0049505
    history = np.tile(np.arange(V, dtype=np.int32)[:L], (B, 1))
    c = lambda a: torch.as_tensor(a).cuda()  # noqa: E731
    lens = c(np.full(B, L, np.int32))
    got = svp.adjust_logits(c(x), history=c(history), history_lens=lens, prompt_lens=lens, repetition=c(r))
    y = got["logits"].double().cpu().numpy()[:, 0]
    want = x[:, 0].astype(np.float64)
    want[:, :L] /= r[:, None].astype(np.float64)
    off = np.abs(y / want - 1)
    assert off.max() <= 2.0**-23 + 2.0**-47
    assert (off[:, L:] == 0).all()

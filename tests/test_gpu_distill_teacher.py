"""Teachers' values far from log probabilities: any constant added under
TAIL_RENORM, masses past the range of 32 bits under TAIL_BUCKET."""

import numpy as np
import pytest
import torch

import vocab_reference as ref
from test_gpu_distill import _case, _grad_ok

pytestmark = pytest.mark.gpu


def _svp():
    import speculative_decoding_verification_60_gb300 as svp

    return svp


@pytest.mark.parametrize("V", [700, 50021])
@pytest.mark.parametrize("constant", [-1e6, -3000.0, 0.0, 50.0, 20000.0, 3e6])
def test_a_constant_added_to_the_teacher(V, constant):
    """Raw logits, say: t_j goes by differences of the values, which are exact or off by their own last bit."""
    svp = _svp()
    K = 9
    s, ids, l = _case(6, V, K, "f32", seed=V)
    l = (l * 3 + constant).float()  # with a constant of 3e6 in steps of a quarter
    a = (s.cuda(), ids.cuda(), l.cuda())
    got = svp.distill_topk(*a, tail=svp.TAIL_RENORM)
    back = svp.distill_topk_backward(*a, got["row_stats"])["grad"].double().cpu().numpy()
    grad, loss = got["grad"].double().cpu().numpy(), got["loss"].double().cpu().numpy()
    assert int(got["dev_error"]) == 0
    for r in range(6):
        i, lr, sr = ids[r].numpy(), l[r].numpy(), s[r].numpy()
        want, g, scale, err = ref.distill_row(sr, i, lr, 1.0, False)
        spread = lr - lr.max()
        assert err == 0 and abs(loss[r] - want) <= ref.distill_loss_bound(sr, i, spread, 1.0)
        far = float(np.abs(spread).max()) + 40.0
        for h in (grad[r], back[r]):
            _grad_ok(h, g, scale, i, lr, V, 1.0, 1.0, "f32", far)


@pytest.mark.parametrize("V", [700, 128256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_teacher_whose_mass_no_float_holds(V, dtype):
    svp = _svp()
    s, ids, l = _case(5, V, 6, dtype, seed=V)
    l[1, 2] = 89.0
    l[2, :] = 88.5  # none of them alone
    l[3, 5] = 1e5
    a = (s.cuda(), ids.cuda(), l.cuda())
    got = svp.distill_topk(*a, tail=svp.TAIL_BUCKET)
    alone = svp.distill_topk(*a, tail=svp.TAIL_BUCKET, with_grad=False)
    back = svp.distill_topk_backward(*a, got["row_stats"])
    assert int(got["dev_error"]) == int(alone["dev_error"]) == ref.DEVERR_NONFINITE
    for r in (1, 2, 3):
        assert float(got["loss"][r]) == 0 == float(alone["loss"][r])
        assert not got["grad"][r].any() and not back["grad"][r].any()
    for r in (0, 4):
        assert float(got["loss"][r]) > 0 and got["grad"][r].any()

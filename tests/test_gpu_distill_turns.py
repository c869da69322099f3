"""spec_distill_topk with more rows than CTAs or clusters run at once: each
takes several in turn, and rows of weight zero and refused rows lie between
them."""

import numpy as np
import pytest
import torch

import vocab_reference as ref
from test_gpu_distill import DTYPE, _grad_ok

pytestmark = pytest.mark.gpu


def _rows(R, V, K, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = torch.empty(R, V, dtype=DTYPE[dtype], device="cuda")
    ids, l = torch.empty(R, K, dtype=torch.int32, device="cuda"), torch.empty(R, K, device="cuda")
    for r in range(0, R, 64):
        x = torch.randn(min(64, R - r), V, generator=g, device="cuda") * 2
        top = torch.log_softmax(x, 1).topk(K, dim=1)
        l[r:r + 64], ids[r:r + 64] = top.values, top.indices.to(torch.int32)
        s[r:r + 64] = (x + 0.7 * torch.randn(x.shape, generator=g, device="cuda")).to(s.dtype)
    return s, ids, l


# V: CTAs that share a row (1, 2, 4, 8, 16); R: several turns of each; once: rows that are all taken in the first turn
@pytest.mark.parametrize("V,dtype,R,once", [(9000, "bf16", 1400, 400), (9001, "f32", 1000, 400), (40003, "bf16", 800, 200),
                                            (20011, "f32", 800, 200), (128256, "bf16", 460, 100), (50021, "f32", 460, 100),
                                            (262144, "bf16", 200, 40), (131075, "f32", 200, 40), (524280, "f32", 36, 6)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_of_every_turn(V, dtype, R, once, in_place):
    import speculative_decoding_verification_60_gb300 as svp

    K = 20
    s, ids, l = _rows(R, V, K, dtype, seed=V + R)
    rng = np.random.default_rng(R)
    w = torch.rand(R, device="cuda") + 0.5
    zero = rng.choice(R, R // 7, replace=False)
    w[torch.as_tensor(zero).cuda()] = 0.0
    live = np.setdiff1d(np.arange(R), zero)
    bad = rng.choice(live, R // 11, replace=False)
    s[torch.as_tensor(bad).cuda(), V // 3] = float("nan")
    s[torch.as_tensor(zero[:3]).cuda()] = float("nan")  # not read
    parts = []
    for r in range(0, R, once):
        o = svp.distill_topk(s[r:r + once], ids[r:r + once], l[r:r + once], w[r:r + once], 1.3)
        parts.append((o["loss"], o["row_stats"], o["grad"]))
    one = [torch.cat(p) for p in zip(*parts)]
    rows = rng.choice(np.setdiff1d(live, bad), 12, replace=False)
    x = s[torch.as_tensor(rows).cuda()].float().cpu().numpy()
    out = svp.distill_topk(s, ids, l, w, 1.3, out=dict(grad=s) if in_place else {})
    assert int(out["dev_error"]) == ref.DEVERR_NONFINITE
    # the same bits as in the first turn
    assert torch.equal(out["loss"], one[0]) and torch.equal(out["row_stats"], one[1])
    assert torch.equal(out["grad"].view(torch.uint8), one[2].view(torch.uint8))
    for r in (*zero, *bad):
        assert float(out["loss"][r]) == 0 and not out["grad"][r].any()
    for k, r in enumerate(rows):
        i, lr, wr = ids[r].cpu().numpy(), l[r].cpu().numpy(), float(w[r])
        loss, g, scale, err = ref.distill_row(x[k], i, lr, 1.3, True)
        assert err == 0 and abs(float(out["loss"][r]) - loss) <= ref.distill_loss_bound(x[k], i, lr, 1.3)
        far = min(200.0, float(np.abs(lr).max()) + 40.0)
        _grad_ok(out["grad"][r].double().cpu().numpy(), g, scale, i, lr, V, 1.3, wr, dtype, far)


@pytest.mark.parametrize("R,V", [(2000, 5000), (1500, 40003)])
def test_the_loss_of_many_rows(R, V):
    import speculative_decoding_verification_60_gb300 as svp

    s, ids, l = _rows(R, V, 128, "bf16", seed=R)
    w = torch.ones(R, device="cuda")
    w[::5] = 0.0
    s[::5] = float("nan")
    out = svp.distill_topk(s, ids, l, w, with_grad=False)
    assert int(out["dev_error"]) == 0 and not out["loss"][::5].any()
    for r in np.random.default_rng(R).choice(R, 20, replace=False):
        if r % 5:
            x, i, lr = s[r].float().cpu().numpy(), ids[r].cpu().numpy(), l[r].cpu().numpy()
            loss = ref.distill_row(x, i, lr, 1.0, True)[0]
            assert abs(float(out["loss"][r]) - loss) <= ref.distill_loss_bound(x, i, lr, 1.0)

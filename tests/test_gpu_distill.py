"""spec_distill_topk and its backward call against the 64-bit reference,
with bounds from the 32-bit sums and the gradient type's rounding."""

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


def _case(R, V, K, dtype, seed, sigma=0.7):
    teacher = synth.zipf_logits(R, V, seed).float() + synth.gaussian((R, V), 0.01, seed + 1)
    lp = torch.log_softmax(teacher.double(), 1).float()
    l, ids = lp.topk(K, dim=1)
    s = (teacher + synth.gaussian((R, V), sigma, seed + 2)).to(DTYPE[dtype])
    return s, ids.to(torch.int32), l


def _grad_ok(g, want, scale, ids, l, V, T, w, dtype, far):
    # each term q or t is off by the sums' bound and the rounding of its exponent (8 units per unit of it)
    rel = ref.sum_bound(V) + ref.EPS * 8 * (len(ids) + far)
    rnd = 2.0 ** -8 if dtype == "bf16" else 2 * ref.EPS  # half a unit in the last of 8 bits
    # exponentials and results below the smallest normal number are flushed; the former are scaled by up to 2 |w| / T
    tiny = 2.0 ** -126 * (1 + 2 * abs(w) / T)
    tol = abs(w) * scale * rel + rnd * np.abs(w * want) + tiny
    bad = np.abs(g - w * want) > tol
    assert not bad.any(), (np.abs(g - w * want)[bad].max(), int(bad.sum()))


def _check(s, ids, l, T, bucket, weights=None, dtype="bf16", placed=None, rows=None, in_place=False):
    svp = _svp()
    R, V = s.shape
    dev = placed if placed is not None else s.cuda()
    out = dict(grad=dev) if in_place else {}
    w = None if weights is None else torch.as_tensor(weights, dtype=torch.float32).cuda()
    tail = svp.TAIL_BUCKET if bucket else svp.TAIL_RENORM
    a = (ids.cuda(), l.cuda())
    alone = svp.distill_topk(dev, *a, w, T, tail, with_grad=False)
    back = svp.distill_topk_backward(dev, *a, alone["row_stats"], w, T)["grad"]
    got = svp.distill_topk(dev, *a, w, T, tail, out=out)
    losses = [o["loss"].cpu().numpy().astype(np.float64) for o in (got, alone)]
    loss = losses[0]
    grad = got["grad"].double().cpu().numpy()
    back = back.double().cpu().numpy()
    bits = 0
    for r in (range(R) if rows is None else rows):
        wr = 1.0 if weights is None else float(np.float32(weights[r]))
        if wr == 0:
            assert loss[r] == 0 and not grad[r].any() and not back[r].any()
            continue
        i, lr, sr = ids[r].numpy(), l[r].numpy(), s[r].float().numpy()
        want, g, scale, err = ref.distill_row(sr, i, lr, T, bucket)
        bits |= err
        bound = 0.0 if err else ref.distill_loss_bound(sr, i, lr, T)
        for value in (losses[0][r], losses[1][r]):
            if want + bound < np.finfo(np.float32).max:
                assert abs(value - want) <= bound, (r, value, want)
            else:  # +inf, or at the end of the range of 32 bits
                assert value >= want - bound if np.isfinite(want) else value == want
        far = 0.0 if err else min(200.0, float(np.abs(lr[np.isfinite(lr)]).max(initial=0.0)) + 40.0)
        for h in (grad[r], back[r]):
            _grad_ok(h, g, scale, i, lr, V, T, wr, dtype, far)
    if rows is None:
        assert int(got["dev_error"]) == bits == int(alone["dev_error"])
    return got


@pytest.mark.parametrize("V,K", [(1, 1), (2, 1), (5, 5), (31, 3), (32, 32), (33, 20), (1001, 64), (4097, 128),
                                 (8192, 16), (32000, 16), (50021, 33), (128256, 64), (129280, 128), (262144, 8),
                                 (524280, 20)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bucket", [False, True])
def test_vocabularies(V, K, dtype, bucket):
    s, ids, l = _case(4 if V > 100000 else 8, V, K, dtype, seed=V + K)
    _check(s, ids, l, 1.0, bucket, dtype=dtype)


@pytest.mark.parametrize("R", [1, 2, 37, 38, 39, 77, 153, 400, 1300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_counts(R, dtype):
    s, ids, l = _case(R, 9000, 12, dtype, seed=R)
    rows = sorted(np.random.default_rng(R).choice(R, min(R, 16), replace=False).tolist())
    _check(s, ids, l, 1.0, True, dtype=dtype, rows=rows)


@pytest.mark.parametrize("T", [0.1, 0.7, 2.0, 6.0])
@pytest.mark.parametrize("bucket", [False, True])
def test_temperatures_and_weights(T, bucket):
    s, ids, l = _case(9, 3000, 10, "bf16", seed=3)
    w = np.array([1, 0, 0.25, -2, 3, 0, 1e-3, 1, 0.5])
    _check(s, ids, l, T, bucket, weights=w)


def test_rows_of_weight_zero_are_not_read():
    s, ids, l = _case(3, 3000, 10, "bf16", seed=4)
    s[1] = float("nan")
    ids[1] = 12345678
    got = _check(s, ids, l, 1.0, True, weights=np.array([1.0, 0.0, 1.0]))
    assert int(got["dev_error"]) == 0


@pytest.mark.parametrize("V,pad,offset", [(1000, 0, 1), (1001, 0, 0), (1001, 7, 3), (4096, 5, 2), (50000, 24, 8),
                                          (9, 1, 5), (128256, 3, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("in_place", [False, True])
def test_strides_alignment_and_in_place(V, pad, offset, dtype, in_place):
    s, ids, l = _case(5, V, min(V, 9), dtype, seed=V)
    buf = torch.full((offset + 5 * (V + pad),), 77.0, dtype=s.dtype, device="cuda")
    rows = buf[offset:].view(5, V + pad)[:, :V]
    rows.copy_(s)
    _check(s, ids, l, 1.0, True, dtype=dtype, placed=rows, in_place=in_place)
    # nothing outside the rows is written
    around = buf[offset:].view(5, V + pad)[:, V:]
    assert (around == 77.0).all() and (buf[:offset] == 77.0).all()


def test_gradient_rows_of_another_alignment():
    svp = _svp()
    s, ids, l = _case(5, 5000, 9, "bf16", seed=6)
    buf = torch.full((3 + 5 * 5005,), 7.0, dtype=s.dtype, device="cuda")
    grad = buf[3:].view(5, 5005)[:, :5000]
    got = svp.distill_topk(s.cuda(), ids.cuda(), l.cuda(), out=dict(grad=grad))
    want = svp.distill_topk(s.cuda(), ids.cuda(), l.cuda())
    assert torch.equal(got["grad"], want["grad"]) and (buf[:3] == 7).all()
    back = svp.distill_topk_backward(s.cuda(), ids.cuda(), l.cuda(), want["row_stats"], out=dict(grad=grad.zero_()))
    assert torch.allclose(back["grad"].float(), want["grad"].float(), rtol=2 ** -7, atol=1e-12)


@pytest.mark.parametrize("bucket", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_absent_and_impossible_teacher_entries(bucket, dtype):
    s, ids, l = _case(7, 2000, 8, dtype, seed=7)
    ids[0, 3:] = -1
    ids[1] = -1  # no teacher at all
    l[2, 1:] = -float("inf")
    l[3] = -float("inf")  # listed, but all of probability zero
    ids[4, ::2] = -1
    l[4, ::2] = float("nan")  # not looked at
    l[5] += 0.0 if bucket else 50.0  # RENORM takes any constant
    got = _check(s, ids, l, 1.0, bucket, dtype=dtype)
    assert int(got["dev_error"]) == 0


@pytest.mark.parametrize("V", [300, 50021, 128256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bucket", [False, True])
def test_masks(V, dtype, bucket):
    K = 12
    s, ids, l = _case(7, V, K, dtype, seed=V)
    low = torch.finfo(DTYPE[dtype]).min
    listed = torch.zeros(7, V, dtype=torch.bool).scatter_(1, ids.long(), True)
    s[0][~listed[0]] = -float("inf")  # the student rules out all but the listed tokens
    s[1][~listed[1]] = low
    s[2, ids[2, 4].long()] = -float("inf")  # one of the teacher's tokens is ruled out: loss +inf
    s[3] = low  # all the same lowest value
    s[4][listed[4]] = low  # the listed tokens only
    s[5][~listed[5]] -= 200.0  # a tail that underflows against the row's maximum
    l[0] = torch.log_softmax(l[0], 0)
    got = _check(s, ids, l, 1.0, bucket, dtype=dtype)
    assert int(got["dev_error"]) == 0 and not torch.isnan(got["grad"]).any()
    assert float(got["loss"][2]) == float("inf") and np.isfinite(float(got["loss"][0]))


def test_refused_rows_and_their_neighbours():
    V = 3001
    s, ids, l = _case(9, V, 6, "bf16", seed=9)
    ids[1, 2] = V
    ids[2, 0] = -2
    ids[3, 5] = ids[3, 1]
    s[4, 17] = float("nan")
    s[5, V - 1] = float("inf")
    s[6] = -float("inf")
    l[7, 1] = float("nan")
    assert int(_check(s, ids, l, 1.0, True)["dev_error"]) == 3
    ok = [0, 8]
    assert int(_check(s[ok], ids[ok], l[ok], 1.0, True)["dev_error"]) == 0


def test_gradient_against_differences():
    """The loss itself, moved along random directions: the directional
    derivative is the gradient's product with the direction."""
    svp = _svp()
    s, ids, l = _case(6, 700, 9, "f32", seed=10)
    w = torch.rand(6) + 0.5
    for tail in (svp.TAIL_BUCKET, svp.TAIL_RENORM):
        g = svp.distill_topk(s.cuda(), ids.cuda(), l.cuda(), w.cuda(), 1.3, tail)["grad"].double().cpu()
        for seed in range(4):
            d = synth.gaussian((6, 700), 1.0, 50 + seed)
            h = 2.0 ** -6
            f = [svp.distill_topk((s + k * h * d).cuda(), ids.cuda(), l.cuda(), w.cuda(), 1.3, tail,
                                  with_grad=False)["loss"].double().cpu() for k in (-1, 1)]
            slope = (w.double() * (f[1] - f[0])).sum() / (2 * h)
            # third derivatives of a log softmax are below 1 along unit logits: h^2 |d|^3 terms; fp32 losses / h
            tol = 6 * (h * h * 4.0 + 2 * ref.distill_loss_bound(s[0].numpy(), ids[0].numpy(), l[0].numpy(), 1.3) / h)
            assert abs(float(slope - (g * d).sum())) < tol


def test_leading_shape_optional_outputs_and_no_rows():
    svp = _svp()
    s, ids, l = _case(6, 640, 5, "bf16", seed=11)
    flat = svp.distill_topk(s.cuda(), ids.cuda(), l.cuda())
    lead = svp.distill_topk(s.cuda().view(2, 3, 640), ids.cuda().view(2, 3, 5), l.cuda().view(2, 3, 5))
    assert lead["grad"].shape == (2, 3, 640) and torch.equal(lead["grad"].flatten(), flat["grad"].flatten())
    e = svp.distill_topk(s[:0].cuda(), ids[:0].cuda(), l[:0].cuda())
    assert e["loss"].shape == (0,) and e["grad"].shape == (0, 640) and int(e["dev_error"]) == 0


def test_offsets_past_32_bits():
    V, stride = 1000, 2**31 + 8
    s, ids, l = _case(2, V, 6, "bf16", seed=12)
    buf = torch.empty(stride + V, dtype=torch.bfloat16, device="cuda")
    rows = buf.as_strided((2, V), (stride, 1))
    rows.copy_(s)
    _check(s, ids, l, 1.0, True, placed=rows, in_place=True)


def test_same_bits_every_time_and_on_another_stream():
    svp = _svp()
    s, ids, l = (t.cuda() for t in _case(20, 128256, 20, "bf16", seed=13))
    first = svp.distill_topk(s, ids, l)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = svp.distill_topk(s, ids, l, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for k in first:
        assert torch.equal(first[k], again[k]), k

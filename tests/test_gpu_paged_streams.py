"""The calls around the attention on a stream of the caller's, while the current one has other work: what they compute is
what they compute on the current one."""

import pytest
import torch

import test_gpu_adjust
import test_gpu_append
import test_gpu_keep

pytestmark = pytest.mark.gpu


def _svp():
    import speculative_decoding_verification_60_gb300 as svp

    return svp


def on_a_stream(call):
    """call(stream) there, while the current stream multiplies matrices."""
    torch.cuda.synchronize()
    stream, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        busy = busy @ busy * 1e-3
    got = call(stream)
    stream.synchronize()
    return got


@pytest.mark.parametrize("form", ["a new dict", "buffers"])
def test_append(form):
    c = test_gpu_append.make(200, 8, 2, 128, 128, norm=True)
    d = {k: None if t is None else t.cuda() for k, t in c.items()}
    caches = [d["k_cache"].clone(), d["v_cache"].clone()]
    want = _svp().append_kv(**d)
    e = dict(d, k_cache=caches[0], v_cache=caches[1])
    out = None if form == "a new dict" else {k: torch.zeros_like(t) for k, t in want.items()}
    got = on_a_stream(lambda s: _svp().append_kv(**e, out=out, stream=s))
    assert all(torch.equal(got[k], want[k]) for k in ("q", "dev_error"))
    assert torch.equal(caches[0], d["k_cache"]) and torch.equal(caches[1], d["v_cache"])


@pytest.mark.parametrize("form", ["a new dict", "buffers"])
@pytest.mark.parametrize("counts", [None, [4, 0, 2]])
def test_adjust(form, counts):
    c = test_gpu_adjust.make(3, 4, 20011, L=3000, seed=2, counts=counts)
    d = {k: torch.as_tensor(t).contiguous().cuda() for k, t in c.items() if t is not None}
    want = _svp().adjust_logits(**d)
    out = None if form == "a new dict" else {k: torch.zeros_like(t) for k, t in want.items()}
    got = on_a_stream(lambda s: _svp().adjust_logits(**d, out=out, stream=s))
    assert all(torch.equal(got[k], want[k]) for k in ("logits", "dev_error"))


def test_keep():
    lens, accepted, table, path, blocks = test_gpu_keep.make(4, 6, 30, 16, [0, 1, 37, 64], [5, 0, 3, 4])
    caches = [torch.randn(blocks, 16, 2, 64, device="cuda") for _ in range(6)]
    others = [c.clone() for c in caches]
    args = [torch.as_tensor(a).cuda() for a in (path, accepted, lens, table)]
    assert int(_svp().keep_path(caches, *args)["dev_error"]) == 0
    got = on_a_stream(lambda s: _svp().keep_path(others, *args, stream=s))
    assert int(got["dev_error"]) == 0 and all(torch.equal(c, o) for c, o in zip(caches, others))

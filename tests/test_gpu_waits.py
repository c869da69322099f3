"""Waits that run out in the calls over vocabulary rows: a library built so
that some threads take their waits for run out.  The call ends, its error word
says so, the rows concerned are refused and the others are what they were."""

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import vocab_reference as ref

pytestmark = pytest.mark.gpu
TIMEOUT = 16
# every fifth row or cluster; one lane of a warp that takes tiles
COPY = "-DSV_LATE_COPY=((blockIdx.x/cluster_size())%5==2&&threadIdx.x==39)"
# one cluster; a lane of such a warp, and one of the warp that has the loss
CLUSTER = "-DSV_LATE_CLUSTER=(blockIdx.x/cluster_size()==3&&(threadIdx.x==39||threadIdx.x==260))"


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    """The package's calls with either library."""
    import speculative_decoding_verification_60_gb300 as svp
    from speculative_decoding_verification_60_gb300 import _binding, build

    build.build()
    own = svp.load()
    tmp = tmp_path_factory.mktemp("late")
    units = {"copy": [("logprobs", COPY), ("distill", COPY)], "cluster": [("distill", CLUSTER)]}

    def compile_unit(job):
        kind, (name, flag) = job
        obj = str(tmp / f"{kind}_{name}.o")
        subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, flag, "-c", os.path.join(build.CSRC, name + ".cu"), "-o",
                        obj], check=True, capture_output=True)
        return kind, name, obj

    with ThreadPoolExecutor(4) as ex:
        built = list(ex.map(compile_unit, [(k, u) for k, us in units.items() for u in us]))
    libs = {}
    for kind in units:
        changed = {name: obj for k, name, obj in built if k == kind}
        objs = [changed.get(src[:-3], os.path.join(build.BUILD, src[:-3] + ".o")) for src in build.SOURCES]
        libs[kind] = str(tmp / f"{kind}.so")
        subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", libs[kind], *objs], check=True, capture_output=True)
    path = _binding.LIB_PATH

    def use(kind):
        _binding._lib, _binding.LIB_PATH = None, libs[kind]
        svp.load()

    def back():
        _binding._lib, _binding.LIB_PATH = own, path

    def call(kind, f):
        use(kind)
        try:
            return f(svp)
        finally:
            back()

    yield svp, call
    back()


def _rows(R, V, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(R, V, generator=g, device="cuda") * 2).bfloat16()
    return x, torch.randint(0, V, (R,), generator=g, device="cuda").to(torch.int32)


@pytest.mark.parametrize("R,V", [(300, 30000), (90, 128256), (8, 128256), (40, 128256)])
@pytest.mark.parametrize("K", [0, 20])
def test_log_probabilities_whose_copy_is_late(late, R, V, K):
    svp, call = late
    x, tok = _rows(R, V, R)
    want = svp.token_logprobs(x, tok, 1.0, K)
    got = call("copy", lambda lib: lib.token_logprobs(x, tok, 1.0, K))
    assert int(got["dev_error"]) == TIMEOUT | ref.DEVERR_NONFINITE and int(want["dev_error"]) == 0
    bad = torch.arange(R, device="cuda") % 5 == 2
    for k in ("logprob", "rank", "entropy", "top_ids", "top_logprobs"):
        assert torch.equal(got[k][~bad], want[k][~bad]), k
    assert (got["logprob"][bad] == -float("inf")).all() and (got["rank"][bad] == -1).all()
    assert not got["entropy"][bad].any() and (got["top_ids"][bad] == -1).all()


def _teacher(x, K=20):
    top = torch.log_softmax(x.float() + 0.5, 1).topk(K, dim=1)
    return top.indices.to(torch.int32), top.values


@pytest.mark.parametrize("R,V", [(500, 30000), (20, 128256)])
def test_losses_whose_copy_is_late(late, R, V):
    svp, call = late
    x, _ = _rows(R, V, R)
    a = (x, *_teacher(x))
    want = svp.distill_topk(*a, with_grad=False)
    got = call("copy", lambda lib: lib.distill_topk(*a, with_grad=False))
    assert int(got["dev_error"]) == TIMEOUT | ref.DEVERR_NONFINITE
    bad = torch.arange(R, device="cuda") % 5 == 2
    assert torch.equal(got["loss"][~bad], want["loss"][~bad]) and not got["loss"][bad].any()


@pytest.mark.parametrize("R,V", [(1300, 20000), (300, 128256)])
def test_gradients_whose_copy_is_late(late, R, V):
    svp, call = late
    x, _ = _rows(R, V, R)
    a = (x, *_teacher(x))
    want = svp.distill_topk(*a)
    got = call("copy", lambda lib: lib.distill_topk(*a))
    assert int(got["dev_error"]) == TIMEOUT | ref.DEVERR_NONFINITE
    bad = got["loss"] == 0
    assert bad[2] and bad[7] and 0.1 < float(bad.float().mean()) < 0.3
    assert torch.equal(got["loss"][~bad], want["loss"][~bad]) and torch.equal(got["grad"][~bad], want["grad"][~bad])
    assert not got["grad"][bad].any()


def test_an_exchange_that_is_late(late):
    """The cluster's other warps then wait in vain for its next row."""
    svp, call = late
    R, V = 400, 128256
    x, _ = _rows(R, V, 1)
    a = (x, *_teacher(x))
    want = svp.distill_topk(*a)
    got = call("cluster", lambda lib: lib.distill_topk(*a))
    torch.cuda.synchronize()
    assert int(got["dev_error"]) == TIMEOUT | ref.DEVERR_NONFINITE
    bad = torch.nonzero(got["loss"] == 0).flatten().tolist()
    assert len(bad) > 2 and bad[0] == 3 and len({b - a for a, b in zip(bad, bad[1:])}) == 1
    ok = torch.ones(R, dtype=torch.bool, device="cuda")
    ok[bad] = False
    assert torch.equal(got["loss"][ok], want["loss"][ok]) and torch.equal(got["grad"][ok], want["grad"][ok])
    assert not got["grad"][bad[1:]].any()
    b = [t[:20] for t in a]
    want = svp.distill_topk(*b, with_grad=False)
    got = call("cluster", lambda lib: lib.distill_topk(*b, with_grad=False))
    assert int(got["dev_error"]) == TIMEOUT | ref.DEVERR_NONFINITE
    ok = torch.arange(20, device="cuda") != 3
    assert float(got["loss"][3]) == 0 and torch.equal(got["loss"][ok], want["loss"][ok])

"""Waits that run out in the tree attention: a library built so that some threads take their waits for run out.  The call
ends, its error word says so, and the calls after it are as ever."""

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

pytestmark = pytest.mark.gpu
# a thread of: the softmax's warpgroups, the keys' copies, the products, the values' copies, the mending
WHO = {"softmax": 39, "other softmax": 200, "keys": 260, "products": 300, "values": 330, "mending": 370}


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    import speculative_decoding_verification_60_gb300 as svp
    from speculative_decoding_verification_60_gb300 import _binding, build

    build.build()
    own, path = svp.load(), _binding.LIB_PATH
    tmp = tmp_path_factory.mktemp("late")

    def make(item):
        name, thread = item
        obj, lib = str(tmp / f"{thread}.o"), str(tmp / f"{thread}.so")
        flag = f"-DSV_LATE_ATTEND=(blockIdx.x%3==1&&threadIdx.x=={thread})"
        subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, flag, "-c", os.path.join(build.CSRC, "attend.cu"), "-o",
                        obj], check=True, capture_output=True)
        objs = [obj if src == "attend.cu" else os.path.join(build.BUILD, src[:-3] + ".o") for src in build.SOURCES]
        subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", lib, *objs], check=True, capture_output=True)
        return name, lib

    with ThreadPoolExecutor(len(WHO)) as ex:
        libs = dict(ex.map(make, WHO.items()))

    def call(name, f):
        _binding._lib, _binding.LIB_PATH = None, libs[name]
        svp.load()
        try:
            return f()
        finally:
            _binding._lib, _binding.LIB_PATH = own, path

    yield svp, call
    _binding._lib, _binding.LIB_PATH = own, path


@pytest.mark.parametrize("longest", [2000, 40000])
@pytest.mark.parametrize("N,heads", [(3, 4), (60, 8)])
@pytest.mark.parametrize("who", list(WHO))
def test_late(late, who, N, heads, longest):
    """Copies into a ring that is still empty wait for nothing: with a tile or two a CTA (2000) no key's copy is late."""
    svp, call = late
    g = torch.Generator(device="cuda").manual_seed(N)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    B, page = 6, 16
    lens = torch.tensor([900, 10, longest, 0, 300, 64], dtype=torch.int32, device="cuda")
    M = (longest + N) // page + 1
    table = torch.randperm(B * M, generator=g, device="cuda").to(torch.int32).view(B, M)
    q, k, v = rand(B, N, heads, 128), rand(B * M, page, 2, 128), rand(B * M, page, 2, 128)
    run = lambda: svp.tree_attention(q, k, v, table, lens)  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    got = call(who, run)
    torch.cuda.synchronize()
    expect = 0 if longest == 2000 and who in ("keys", "values") else 16
    assert int(want["dev_error"]) == 0 and int(got["dev_error"]) == expect
    again = run()
    assert int(again["dev_error"]) == 0 and torch.equal(again["out"], want["out"])

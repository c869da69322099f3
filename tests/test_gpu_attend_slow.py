"""Roles of the tree attention that come late: a library built so that in every group of CTAs another role (or another
single warp) loses 20 us before each of its waits.  What it computes is what the library computes, bit for bit: no role
counts on another one's pace."""

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from test_gpu_attend import make, on_gpu

pytestmark = pytest.mark.gpu
# two warpgroups of the softmax and four warps (keys, products, values, mending); or each of the twelve warps
WHO = {"a role": "((threadIdx.x<256?threadIdx.x/128:threadIdx.x/32-6)==blockIdx.x/8%6?20000:0)",
       "a warp": "(threadIdx.x/32==blockIdx.x/8%12?20000:0)"}


@pytest.fixture(scope="module")
def slow(tmp_path_factory):
    import speculative_decoding_verification_60_gb300 as svp
    from speculative_decoding_verification_60_gb300 import _binding, build

    build.build()
    own, path = svp.load(), _binding.LIB_PATH
    tmp = tmp_path_factory.mktemp("slow")

    def build_one(item):
        name, late = item
        obj, lib = str(tmp / f"{name[2:]}.o"), str(tmp / f"{name[2:]}.so")
        subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, f"-DSV_SLOW_ATTEND={late}", "-c",
                        os.path.join(build.CSRC, "attend.cu"), "-o", obj], check=True, capture_output=True)
        objs = [obj if src == "attend.cu" else os.path.join(build.BUILD, src[:-3] + ".o") for src in build.SOURCES]
        subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", lib, *objs], check=True, capture_output=True)
        return name, lib

    with ThreadPoolExecutor(len(WHO)) as ex:
        libs = dict(ex.map(build_one, WHO.items()))

    def call(name, f):
        _binding._lib, _binding.LIB_PATH = None, libs[name]
        svp.load()
        try:
            return f()
        finally:
            _binding._lib, _binding.LIB_PATH = own, path

    yield svp, call
    _binding._lib, _binding.LIB_PATH = own, path


def alike(slow, who, c):
    svp, call = slow
    d = on_gpu(c)
    want = svp.tree_attention(**d)
    torch.cuda.synchronize()
    assert int(want["dev_error"]) == 0
    got = call(who, lambda: svp.tree_attention(**d))
    torch.cuda.synchronize()
    assert int(got["dev_error"]) == 0
    assert torch.equal(torch.nan_to_num(got["out"], nan=9.0), torch.nan_to_num(want["out"], nan=9.0))


@pytest.mark.parametrize("who", list(WHO))
@pytest.mark.parametrize("N,heads,kv,dim", [(3, 8, 8, 64), (2, 32, 8, 128), (32, 64, 8, 64), (32, 64, 8, 128)])
@pytest.mark.parametrize("longest", [100, 700])
def test_many_items(slow, who, N, heads, kv, dim, longest):
    """Runs of many items; of sequences of several tiles, so that runs end within items, some of them after one tile."""
    rng = np.random.default_rng(longest)
    c = make(100, N, heads, kv, dim, 16, rng.integers(0, longest, 100), seed=N + dim)
    nan_in_nodes(c, (3, 4, 5, 40, 70))
    alike(slow, who, c)


def nan_in_nodes(c, requests):
    """What the mending finds must not be lost: in the last node of these requests, if they have one."""
    N, kv = c["q"].shape[1], c["k_cache"].shape[2]
    for b in requests:
        n = N if c["n_nodes"] is None else int(c["n_nodes"][b])
        t = int(c["seq_lens"][b]) + n - 1
        if n > 0:
            c["v_cache"][int(c["block_table"][b, t // 16]), t % 16, b % kv, 7] = float("nan")


@pytest.mark.parametrize("who", list(WHO))
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("longest", [60, 700])
@pytest.mark.parametrize("nodes", ["33", "1 to 16", "16 or 17", "0 to 40"])
def test_empty_second_blocks(slow, who, dim, longest, nodes):
    """Items whose second block of rows is empty: always, in a share's CTAs alone, and now and then."""
    rng = np.random.default_rng(dim + longest)
    B, counts = 120, dict([("33", None), ("1 to 16", rng.integers(1, 17, 120)), ("16 or 17", rng.integers(16, 18, 120)),
                           ("0 to 40", rng.integers(0, 41, 120))])[nodes]
    N = {"33": 33, "1 to 16": 32, "16 or 17": 32, "0 to 40": 40}[nodes]
    c = make(B, N, 64, 8, dim, 16, rng.integers(0, longest, B), form="dynamic", counts=counts, seed=dim)
    nan_in_nodes(c, range(3, B, 7))
    alike(slow, who, c)

"""append_kv against the definition in 64 bits: types, layouts, turned parts of a head, norms, far positions, slots."""

import numpy as np
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu


def _svp():
    import speculative_decoding_verification_60_gb300 as svp

    return svp


def make(T, heads, kv, dim, rot, dtype=torch.bfloat16, page=16, last=5000, norm=False, by_head=False, fused=True, seed=0,
         skip=0.2, theta=10000.0):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    qkv = torch.randn(T, heads + 2 * kv, dim, generator=g).to(dtype)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    blocks = -(-T // page) + 2
    slots = torch.tensor(rng.permutation(blocks * page)[:T], dtype=torch.int64)
    slots[torch.rand(T, generator=g) < skip] = -1
    shape = (blocks, kv, page, dim) if by_head else (blocks, page, kv, dim)
    caches = [torch.randn(shape, generator=g).to(dtype) for _ in range(2)]
    if by_head:
        caches = [c.transpose(1, 2) for c in caches]
    positions = torch.randint(0, last + 1, (T,), generator=g).to(torch.int32)
    positions[0] = last
    inv_freq = torch.tensor([theta ** (-2.0 * i / max(rot, 1)) for i in range(rot // 2)]) if rot else None
    norms = [(torch.randn(dim, generator=g) * 0.2 + 1).to(dtype) for _ in range(2)] if norm else [None, None]
    return dict(q=q, k=k, v=v, positions=positions, slots=slots, k_cache=caches[0], v_cache=caches[1], inv_freq=inv_freq,
                q_norm=norms[0], k_norm=norms[1])


def near(got, want, size, dtype):
    """One rounding to the type, and before it 32 bits: sines, cosines and the angle to 2^-22 of the pair's size, the
    norm's sum and root to 2^-18 of it."""
    u = ref.half_step(dtype)
    tiny = torch.finfo(dtype).smallest_normal * u * 2
    assert bool(((got.double().cpu() - want).abs() <= want.abs() * u * 1.01 + size * 2.0**-17 + tiny).all())


def run(c, interleaved=False, eps=1e-6, error=0, in_place=False):
    want_q, want_k, stored = ref.append(c["q"], c["k"], c["v"], c["positions"], c["slots"], c["k_cache"], c["v_cache"],
                                        c["inv_freq"], c["q_norm"], c["k_norm"], eps, interleaved)

    def move(t):
        return None if t is None else torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)

    d = {key: move(t) for key, t in c.items()}
    dtype = c["k"].dtype
    for _ in range(1 if in_place else 2):  # the call can be repeated
        out = dict(q=d["q"]) if in_place else None
        got = _svp().append_kv(**d, eps=eps, interleaved=interleaved, out=out)
        assert int(got["dev_error"]) == error
    size = lambda x: x.abs().amax(2, keepdim=True)  # noqa: E731
    if want_q is not None:
        near(got["q"], want_q, size(want_q), dtype)
    page = c["k_cache"].shape[1]
    for name, want in (("k_cache", want_k), ("v_cache", c["v"])):
        expect = c[name].clone().flatten(0, 1) if c[name].is_contiguous() else c[name].reshape(-1, *c[name].shape[2:])
        cache = d[name].cpu().reshape(-1, *c[name].shape[2:])
        others = torch.ones(cache.shape[0], dtype=torch.bool)
        for s, t in stored.items():
            others[s] = False
            if name == "v_cache":
                assert torch.equal(cache[s], want[t])
        assert torch.equal(cache[others], expect[others])
        if name == "k_cache" and stored:
            at, tokens = list(stored.keys()), list(stored.values())
            near(cache[at], want[tokens], size(want[tokens]), dtype)
    assert page > 0
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,rot", [(8, 8), (64, 64), (80, 80), (80, 40), (96, 48), (96, 96), (128, 128), (128, 32),
                                     (256, 256), (256, 64), (64, 0), (24, 16), (104, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads(dtype, dim, rot, interleaved):
    run(make(13, 6, 2, dim, rot, dtype), interleaved)
    run(make(13, 3, 3, dim, rot, dtype, norm=True, seed=1), interleaved, eps=1e-5)


@pytest.mark.parametrize("T", [0, 1, 2, 300])
@pytest.mark.parametrize("heads,kv", [(1, 1), (64, 8), (5, 1)])
def test_tokens(T, heads, kv):
    if T == 0:
        c = make(1, heads, kv, 64, 64)
        d = {key: None if t is None else (t if "cache" in key or key == "inv_freq" else t[:0]).cuda()
             for key, t in c.items()}
        got = _svp().append_kv(**d)
        assert got["q"].shape == (0, heads, 64) and int(got["dev_error"]) == 0
        assert torch.equal(d["k_cache"].cpu(), c["k_cache"])
    else:
        run(make(T, heads, kv, 64, 64))


@pytest.mark.parametrize("last", [0, 1, 100000, 10**7, 2**31 - 1])
@pytest.mark.parametrize("theta", [10000.0, 1e8])
def test_far_positions(last, theta):
    c = make(40, 2, 1, 128, 128, torch.float16, last=last, theta=theta)
    run(c)
    c["positions"] = -c["positions"]
    run(c)


@pytest.mark.parametrize("page,by_head", [(1, False), (7, True), (48, True), (128, False)])
def test_caches(page, by_head):
    run(make(50, 4, 2, 64, 64, page=page, by_head=by_head, fused=False))


def test_narrow_vectors():
    """Strides and pointers on 8 bytes only."""
    c = make(9, 2, 2, 64, 64)
    wide = torch.zeros(9, 2, 68, dtype=torch.bfloat16)
    wide[:, :, 4:] = c["q"]
    c["q"] = wide[:, :, 4:]
    run(c)


def test_in_place():
    run(make(20, 4, 2, 64, 64, fused=False), in_place=True)
    run(make(20, 4, 2, 96, 96, fused=False, norm=True), in_place=True)


def test_keys_and_values_alone():
    c = make(11, 4, 2, 64, 64, norm=True)
    c["q"] = c["q_norm"] = None
    run(c)


def test_slots_that_the_cache_does_not_have():
    c = make(11, 4, 2, 64, 64, skip=0.0)
    entries = c["k_cache"].shape[0] * 16
    c["slots"][3], c["slots"][7], c["slots"][9] = entries, 2**62, -(2**62)
    run(c, error=32)


def test_values_keep_their_bits():
    """Infinities, NaN and what is not turned or normed pass through."""
    c = make(6, 2, 2, 64, 32, torch.float16, skip=0.0)
    for key in ("q", "k"):
        c[key][:, :, 40] = float("inf")
        c[key][:, :, 41] = 65504.0
    c["v"][:, :, 3] = float("nan")
    d = {key: None if t is None else t.cuda() for key, t in c.items()}
    got = _svp().append_kv(**d)
    assert torch.equal(got["q"][:, :, 32:].cpu(), c["q"][:, :, 32:])
    flat = d["v_cache"].flatten(0, 1)[c["slots"].cuda()].cpu()
    assert torch.equal(flat.view(torch.int16), c["v"].contiguous().view(torch.int16))


def test_a_graph():
    c = make(20, 4, 2, 64, 64)
    d = {key: None if t is None else t.cuda() for key, t in c.items()}
    out = _svp().append_kv(**d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _svp().append_kv(**d, out=out)
    d["positions"].add_(17)
    graph.replay()
    assert torch.equal(out["q"], _svp().append_kv(**d)["q"])

"""How far results of the calls over a paged cache and the logits may be off, as the header states it."""

from fractions import Fraction

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


def turn(position, inv):
    """position * inv modulo a turn, in radians within half a turn of 0, from whole numbers."""
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068423413")
    turns = Fraction(position) * Fraction(float(inv)) / two_pi
    return float((turns - round(turns)) * two_pi)


@pytest.mark.parametrize("theta", [10000.0, 1e8])
def test_angles(theta):
    """The angle to 2^-25.9 turns at any position.  Pairs that are turned to where one of the two nearly vanishes show
    it: fp16 holds 6e4 sin(delta) to 2^-12 and less there."""
    import speculative_decoding_verification_60_gb300 as svp

    rng = np.random.default_rng(8)
    T, D = 400, 128
    inv = np.array([theta ** (-2.0 * i / D) for i in range(D // 2)], np.float32)
    positions = rng.integers(0, 2**31, T)
    positions[:100] = rng.integers(0, 131072, 100)
    angle = np.array([[turn(int(p), f) for f in inv] for p in positions])
    x = np.zeros((T, 1, D))
    x[:, 0, :64], x[:, 0, 64:] = 4e4 * np.sin(angle), 4e4 * np.cos(angle)  # turned, the first is near 0
    k = torch.tensor(x).half()
    cache = [torch.zeros(T, 1, 1, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    got = svp.append_kv(k.cuda(), k.cuda(), k.cuda(), torch.tensor(positions, dtype=torch.int32, device="cuda"),
                        torch.arange(T, device="cuda"), *cache, torch.tensor(inv, device="cuda"))
    assert int(got["dev_error"]) == 0
    a, b = [k.double().numpy()[:, 0, s] for s in (slice(0, 64), slice(64, 128))]
    want = np.concatenate([a * np.cos(angle) - b * np.sin(angle), b * np.cos(angle) + a * np.sin(angle)], 1)
    size = np.hypot(a, b)
    # the angle; sine and cosine to a unit in their last place each (2^-24 below 1); a product rounded to 2^-24; its sum
    # with the other rounded, and the type
    far = size * (2 * np.pi * 2.0**-25.9 + (2**0.5 + 1) * 2.0**-24)
    for turned in (got["q"], cache[0][:, 0]):
        off = np.abs(turned.double().cpu().numpy()[:, 0] - want)
        assert (off <= np.tile(far, 2) + np.abs(want) * (2.0**-11 + 2.0**-24) * 1.01 + 2.0**-25).all()


@pytest.mark.parametrize("pad", [0, 4])  # vectors of 16 bytes, and of 8
def test_a_slot_named_twice(pad):
    """Every 8 bytes of the entry are one of the tokens'; the entries beside it stay."""
    import speculative_decoding_verification_60_gb300 as svp

    g = torch.Generator(device="cuda").manual_seed(9)
    T, H, D = 300, 3, 64
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    k, v = rand(T, H, D + pad)[..., pad:], rand(T, H, D + pad)[..., pad:]
    caches = [rand(4, 8, H, D) for _ in range(2)]
    before = [c.clone() for c in caches]
    got = svp.append_kv(None, k, v, None, torch.full((T,), 13, device="cuda"), *caches)
    assert int(got["dev_error"]) == 0
    for x, cache, old in zip((k, v), caches, before):
        flat, old = cache.flatten(0, 1), old.flatten(0, 1)
        eights = x.contiguous().view(torch.int64)
        assert bool((eights == flat[13].contiguous().view(torch.int64)).any(0).all())
        rest = torch.arange(32, device="cuda") != 13
        assert torch.equal(flat[rest], old[rest])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("at", [0, 19999])
def test_a_long_tail(dtype, at):
    """One dominant entry, first or last, beside 20,000 of 2^-20 of its weight: half a step of the type for each weight,
    and in fp16, where they are subnormal, 2^-25 of the dominant one."""
    import speculative_decoding_verification_60_gb300 as svp

    L, D, page = 20000, 64, 64
    g = torch.Generator().manual_seed(10)
    blocks = L // page + 1
    k = torch.zeros(blocks * page, 1, D, dtype=dtype)
    k[:, 0, 0] = -20 * np.log(2)
    k[at, 0, 0] = 0.0
    v = (torch.rand(blocks * page, 1, D, generator=g) + 0.5).to(dtype)  # of one sign: errors of one sign add up
    q = torch.zeros(1, 1, 2, D, dtype=dtype)
    q[..., 0] = 1.0
    table = torch.arange(blocks, dtype=torch.int32)[None]
    args = [q, k.view(blocks, page, 1, D), v.view(blocks, page, 1, D), table, torch.tensor([L - 1], dtype=torch.int32)]
    got = svp.tree_attention(*[t.cuda() for t in args], scale=1.0)
    assert int(got["dev_error"]) == 0
    s = k[:L, 0, 0].double()
    w = torch.exp(s - s.max())
    want = (w @ v[:L, 0].double()) / w.sum()
    u = torch.finfo(dtype).eps / 2
    # sums of 20,000 terms in 32 bits in an order of the kernel's: at most 2^-24 of the sum a term
    far = (u * want * 2 + L * 2.0**-24 * want) * 1.01
    if dtype is torch.float16:
        far = far + L * 2.0**-25 * v[:L, 0].double().amax(0)
    assert bool(((got["out"][0, 0].double().cpu() - want).abs() <= far).all())

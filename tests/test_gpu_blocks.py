"""spec_advance_blocks against the plain reference: every output equal."""

import numpy as np
import pytest
import torch

import vocab_reference as ref

pytestmark = pytest.mark.gpu


def _svp():
    import speculative_decoding_verification_60_gb300 as svp

    return svp


def _case(B, page, M, most_new, seed, spare=None, cap=None):
    rng = np.random.default_rng(seed)
    room = page * M
    new = rng.integers(0, min(most_new, room) + 1, B)
    acc = rng.integers(-1, 5, B)
    lens = rng.integers(0, np.maximum(1, room - new - 5), B) if room > most_new + 6 else np.zeros(B, np.int64)
    acc = np.where(lens + acc + 1 + new > room, -1, acc)
    held = np.minimum(M, -(-(lens + 5) // page))
    acc = np.where(lens + acc + 1 > held * page, -1, acc)
    blocks = rng.permutation(B * M + 7).astype(np.int32)
    table = np.full((B, M), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = blocks[at:at + held[b]]
        at += held[b]
    free = blocks[at:].copy()
    count = len(free) if spare is None else spare
    i32 = lambda a: np.asarray(a, np.int32)  # noqa: E731
    return i32(lens), i32(acc), i32(new), page, table, i32(held), free, count


def _run(case, max_tokens, accepted=True, stride=None):
    lens, acc, new, page, table, held, free, count = case
    c = lambda a: torch.as_tensor(np.ascontiguousarray(a)).cuda()  # noqa: E731
    t = c(table)
    if stride:
        wide = torch.full((table.shape[0], stride), -9, dtype=torch.int32, device="cuda")
        wide[:, : table.shape[1]] = t
        t = wide[:, : table.shape[1]]
    a = acc if accepted else None
    want, err = ref.advance_blocks(lens, a, new, page, table, held, free, count, max_tokens)
    inputs = (c(lens), c(new), t, c(held), c(free), torch.tensor([count], dtype=torch.int32).cuda())
    for _ in range(2):  # the call can be repeated on the same inputs
        got = _svp().advance_blocks(*inputs, page, max_tokens, accepted_len=None if a is None else c(a))
        for key in ("seq_lens", "held", "cu_tokens", "slots", "positions"):
            assert np.array_equal(got[key].cpu().numpy(), want[key]), key
        assert np.array_equal(t.cpu().numpy(), want["table"])
        assert int(got["free_count"]) == want["free_count"] and int(got["dev_error"]) == err
    if stride:
        assert (wide[:, table.shape[1]:] == -9).all()
    return want, err


@pytest.mark.parametrize("B", [1, 2, 31, 33, 64, 255, 1024, 1025, 2500])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
def test_requests_and_pages(B, page):
    case = _case(B, page, 40, 9, seed=B + page)
    _, err = _run(case, int(case[2].sum()) + 5)
    assert err == 0


@pytest.mark.parametrize("B,most", [(1, 100000), (7, 9000), (300, 4096), (16384, 3)])
def test_long_prompts_and_many_requests(B, most):
    case = _case(B, 128, 1000 if B < 1000 else 8, most, seed=B)
    _, err = _run(case, int(case[2].sum()))
    assert err == 0


def test_without_acceptance_and_without_new_tokens():
    case = _case(50, 16, 20, 6, seed=1)
    _run(case, 300, accepted=False)
    lens, acc, new, *rest = case
    _run((lens, acc, new * 0, *rest), 16)
    _run((lens, acc, new * 0, *rest), 0)


def test_a_table_with_wider_rows():
    _run(_case(20, 16, 20, 6, seed=2), 200, stride=33)


@pytest.mark.parametrize("spare", [0, 1, 5, 17, 60])
def test_a_free_list_that_runs_out(spare):
    case = _case(80, 4, 30, 9, seed=spare, spare=spare)
    want, err = _run(case, 800)
    assert (err == ref.DEVERR_CAPACITY) == (want["slots"][: want["cu_tokens"][-1]] < 0).any()
    assert spare > 20 or err


def test_a_table_row_that_runs_out():
    lens, acc, new, page, table, held, free, count = _case(40, 4, 12, 5, seed=4)
    new[[3, 20]] = 49
    _, err = _run((lens, acc, new, page, table, held, free, count), 400)
    assert err == ref.DEVERR_CAPACITY


def test_more_tokens_than_the_buffer_holds():
    case = _case(40, 4, 12, 5, seed=5)
    _, err = _run(case, int(case[2].sum()) - 3)
    assert err == ref.DEVERR_LENGTH


@pytest.mark.parametrize("count", [-1, 10**9])
def test_a_count_that_is_no_count(count):
    lens, acc, new, page, table, held, free, _ = _case(10, 4, 12, 5, seed=6)
    _, err = _run((lens, acc, new, page, table, held, free, count), 60)
    assert err & ref.DEVERR_LENGTH


def test_malformed_requests_and_their_neighbours():
    lens, acc, new, page, table, held, free, count = _case(40, 4, 12, 5, seed=7)
    lens[1] = -3
    acc[2] = -2
    new[3] = -1
    held[4] = -1
    held[5] = 13
    lens[6], held[6], acc[6] = 40, 2, 0
    lens[7] = 2**31 - 1
    new[8] = 2**31 - 1 - int(new.astype(np.int64).sum()) - 10000  # needs more blocks than a row has
    _, err = _run((lens, acc, new, page, table, held, free, count), 300)
    assert err == ref.DEVERR_LENGTH | ref.DEVERR_CAPACITY


def test_slots_past_32_bits():
    lens, acc, new, page, table, held, free, count = _case(6, 64, 8, 20, seed=8)
    table = np.where(table >= 0, table + 2**30, table).astype(np.int32)
    want, _ = _run((lens, acc, new, page, table, held, free + 2**30, count), 200)
    assert want["slots"].max() > 2**36


def test_after_a_verification():
    """accepted_len and the next call's state, step after step."""
    svp = _svp()
    B, page, M, k = 5, 4, 64, 3
    dev = dict(dtype=torch.int32, device="cuda")
    table = torch.full((B, M), -1, **dev)
    free = torch.randperm(B * M, device="cuda").to(torch.int32)
    lens, held, count = torch.zeros(B, **dev), torch.zeros(B, **dev), torch.tensor([B * M], **dev)
    new = torch.full((B,), k + 1, **dev)
    acc = None
    seen = np.zeros(B, np.int64)
    for step in range(20):
        out = svp.advance_blocks(lens, new, table, held, free, count, page, B * (k + 1), accepted_len=acc)
        lens, held, count = out["seq_lens"], out["held"], out["free_count"]
        assert int(out["dev_error"]) == 0 and np.array_equal(lens.cpu().numpy(), seen)
        used = table[table >= 0]
        assert used.unique().numel() == used.numel() == int(held.sum()) == B * M - int(count)
        acc = torch.randint(0, k + 1, (B,), **dev)
        seen += acc.cpu().numpy() + 1

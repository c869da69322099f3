"""spec_advance_blocks where a buffer for the new tokens reaches the end of
the range of its size."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_tokens", [2**31 - 1, 2**31 - 4])
def test_the_largest_buffers(max_tokens):
    """Every place past the new tokens is -1 or 0, none in front of the
    buffers is written, and the call ends."""
    import speculative_decoding_verification_60_gb300 as svp

    need = (8 + 4) * (2**31 + 64)
    if torch.cuda.mem_get_info()[0] < need + 2**33:
        pytest.skip("needs 34 GB of free memory")
    B, page, M, guard = 3, 16, 4, 16
    i32 = dict(dtype=torch.int32, device="cuda")
    slots = torch.full((guard + max_tokens,), 7, dtype=torch.int64, device="cuda")
    positions = torch.full((guard + max_tokens,), 7, **i32)
    table = torch.full((B, M), -1, **i32)
    free = torch.arange(20, 20 + B * M, **i32)
    out = dict(slots=slots[guard:], positions=positions[guard:])
    new = torch.tensor([5, 17, 3], **i32)
    got = svp.advance_blocks(torch.zeros(B, **i32), new, table, torch.zeros(B, **i32), free,
                             torch.tensor([B * M], **i32), page, max_tokens, out=out)
    assert int(got["dev_error"]) == 0 and got["cu_tokens"].tolist() == [0, 5, 22, 25]
    blocks = table.tolist()
    want = [(b, i) for b, n in enumerate(new.tolist()) for i in range(n)]
    assert got["positions"][:25].tolist() == [i for _, i in want]
    assert got["slots"][:25].tolist() == [blocks[b][i // page] * page + i % page for b, i in want]
    assert (slots[:guard] == 7).all() and (positions[:guard] == 7).all()
    # the rest a part at a time: a mask of all of it would be large, too
    for a in range(25, max_tokens, 2**28):
        assert (got["slots"][a:a + 2**28] == -1).all() and (got["positions"][a:a + 2**28] == 0).all()

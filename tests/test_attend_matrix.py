"""CPU: the two forms of tree_attention's definition say the same."""

import pytest
import torch

import attend_matrix
import paged_reference as ref
from test_gpu_attend import make


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("form,counts", [("chain", None), ("tree", None), ("dynamic", [7, 0, 3, 1])])
def test_alike(dtype, form, counts):
    c = make(4, 7, 6, 2, 24, 8, [19, 0, 40, 3], dtype, form=form, counts=counts, seed=3)
    t = 19 + 6  # a node of the first request
    c["v_cache"][int(c["block_table"][0, t // 8]), t % 8, 1, 5] = float("inf")
    args = [c[x] for x in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "parent", "n_nodes", "scale")]
    (a, x), (b, y) = ref.attend(*args), attend_matrix.attend(*args)
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and bool(torch.isnan(a[0, 6, 3:]).all())
    # sums of up to 47 terms in another order
    assert torch.allclose(a, b, rtol=0, atol=1e-13, equal_nan=True)
    live = ~torch.isnan(a)
    assert torch.allclose(x[live], y[live], rtol=1e-6)

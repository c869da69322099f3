"""tree_attention's definition in 64 bits again (tests/paged_reference.py), by matrices of a request and key head: for
cases of many requests, where a walk over rows takes minutes.  tests/test_attend_matrix.py holds the two together."""

import torch

import paged_reference as ref


def attend(q, k_cache, v_cache, table, lens, parent=None, n_nodes=None, scale=1.0):
    """As paged_reference.attend, for requests that are not refused and sequences whose values are finite."""
    B, N, H, D = q.shape
    heads, page = k_cache.shape[2], k_cache.shape[1]
    group, u = H // heads, ref.half_step(q.dtype)
    out = torch.full((B, N, H, D), float("nan"), dtype=torch.float64)
    bound = torch.zeros_like(out)
    rows = lambda t: t.permute(1, 0, 2, 3).reshape(t.shape[1], N * group, D)[:, :n * group]  # noqa: E731
    for b in range(B):
        n, length = N if n_nodes is None else int(n_nodes[b]), int(lens[b])
        if n == 0:
            continue
        tree = list(range(-1, N - 1)) if parent is None else (parent if parent.dim() == 1 else parent[b]).tolist()
        at = torch.arange(length + n)
        block, place = table[b, at // page].long(), at % page
        k, v = [c[block, place].double().transpose(0, 1) for c in (k_cache, v_cache)]  # [heads, L, D]
        see = torch.zeros(n, length + n, dtype=torch.bool)
        see[:, :length] = True
        for i in range(n):
            see[i, [length + m for m in ref.path(tree, i)]] = True
        see = see.repeat_interleave(group, 0)  # [rows, L]
        x = rows(q[b].double().view(N, heads, group, D))
        s = torch.where(see, scale * (x @ k.transpose(1, 2)), -float("inf"))
        w = torch.exp(s - s.amax(2, keepdim=True))
        total = w.sum(2, keepdim=True)
        finite = torch.isfinite(v).all(2)  # [heads, L]
        known = torch.where(finite[..., None], v, 0.0)
        o = (w @ known) / total
        poisoned = ((~finite).double()[:, None] * see.double()).sum(2) > 0
        spread = (w @ known.abs()) / total
        exponent = torch.where(see, scale * (x.abs() @ k.abs().transpose(1, 2)), 0.0).amax(2, keepdim=True)
        count = see.sum(1).double()[None, :, None]
        sums = 4 * ((D + 8) * exponent + count + 16) * 2.0**-24
        loudest = torch.where(see, known.abs().amax(2)[:, None], 0.0).amax(2, keepdim=True)
        least = count * 2.0**-25 * loudest if q.dtype == torch.float16 else 0.0
        far = u * (spread + o.abs()) * 1.01 + sums * spread + least + (2.0**-25 if u > 2**-12 / 2 else 0)
        o = torch.where(poisoned[..., None], float("nan"), o)
        back = lambda t: t.reshape(heads, n, group, D).transpose(0, 1).reshape(n, H, D)  # noqa: E731
        out[b, :n], bound[b, :n] = back(o), back(far)
    return out, bound

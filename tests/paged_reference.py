"""Definitions of the calls over a paged cache, written out in 64 bits (plain
torch and numpy, on the CPU): what the tests of append_kv, tree_attention,
adjust_logits and keep_path compare with."""

import numpy as np
import torch


def half_step(dtype):
    """The largest rounding error of a value of this type, relative to it."""
    return torch.finfo(dtype).eps / 2


def is_tree(parent):
    return parent[0] == -1 and all(0 <= p < i for i, p in enumerate(parent) if i > 0)


def path(parent, i):
    """Nodes from the root to i."""
    nodes = []
    while i >= 0:
        nodes.append(i)
        i = int(parent[i])
    return nodes[::-1]


def random_tree(n, depth, rng):
    """Parents of a random tree of n nodes, no deeper than depth."""
    level, parent = [0], [-1]
    for i in range(1, n):
        p = int(rng.integers(0, i))
        while level[p] >= depth:
            p = parent[p]
        parent.append(p)
        level.append(level[p] + 1)
    return parent


def turn(x, positions, inv_freq, interleaved):
    """x [T, H, D] in 64 bits, its first 2 len(inv_freq) dimensions turned."""
    half = len(inv_freq)
    angle = positions.double()[:, None] * inv_freq.double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y = x.clone()
    i, j = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def append(q, k, v, positions, slots, k_cache, v_cache, inv_freq, q_norm, k_norm, eps, interleaved):
    """(q', k', {slot: token}) in 64 bits; caches [blocks, page, H, D] are not changed."""

    def one(x, norm):
        x = x.double()
        if norm is not None:
            x = x / (x.square().mean(2, keepdim=True) + eps).sqrt() * norm.double()
        return x if inv_freq is None else turn(x, positions, inv_freq, interleaved)

    stored = {int(s): t for t, s in enumerate(slots.tolist()) if 0 <= s < k_cache.shape[0] * k_cache.shape[1]}
    return None if q is None else one(q, q_norm), one(k, k_norm), stored


def attend(q, k_cache, v_cache, table, lens, parent=None, n_nodes=None, scale=1.0):
    """out [B, N, H, D] in 64 bits (NaN where rows stay as they are), and how far
    a result in q's type may be from it: weights rounded to the type (half a step each),
    the output rounded (half a step), scores and sums in 32 bits."""
    B, N, H, D = q.shape
    heads, page = k_cache.shape[2], k_cache.shape[1]
    u = half_step(q.dtype)
    out = torch.full((B, N, H, D), float("nan"), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for b in range(B):
        n, length = N if n_nodes is None else int(n_nodes[b]), int(lens[b])
        tree = list(range(-1, N - 1)) if parent is None else (parent if parent.dim() == 1 else parent[b]).tolist()
        checked = tree if parent is None or parent.dim() == 1 else tree[:max(n, 0)]
        if n < 0 or n > N or length < 0 or length + n > table.shape[1] * page:
            out[b, :N if n < 0 or n > N else n] = 0
            continue
        blocks = [int(x) for x in table[b, :-(-(length + n) // page)]]
        if (checked and not is_tree(checked)) or (n and any(x < 0 or x >= k_cache.shape[0] for x in blocks)):
            out[b, :n] = 0
            continue
        for i in range(n):
            at = list(range(length)) + [length + m for m in path(tree, i)]
            block = torch.tensor([blocks[t // page] for t in at])
            place = torch.tensor([t % page for t in at])
            k, v = k_cache[block, place].double(), v_cache[block, place].double()  # [L, heads, D]
            for h in range(H):
                g = h // (H // heads)
                x = q[b, i, h].double()
                s = scale * (k[:, g] @ x)
                w = torch.exp(s - s.max())
                total = w.sum()
                o = (w @ v[:, g]) / total
                # a node's entry that is not finite makes the rows that see it NaN
                if not torch.isfinite(v[length:, g]).all():
                    o = torch.full_like(o, float("nan"))
                out[b, i, h] = o
                spread = (w @ v[:, g].abs()) / total
                exponent = scale * float((k[:, g].abs() @ x.abs()).max())
                sums = 4 * ((D + 8) * exponent + len(at) + 16) * 2.0**-24
                least = len(at) * 2.0**-25 * v[:, g].abs().max() if q.dtype == torch.float16 else 0.0
                bound[b, i, h] = u * (spread + o.abs()) * 1.01 + sums * spread + least + (2.0**-25 if u > 2**-12 / 2 else 0)
    return out, bound


def adjust(x, b, i, history, lens, prompt, drafted, parent, repetition, frequency, presence, bias_ids, bias_values,
           allowed):
    """Row i of request b in 64 bits; x its logits, drafted[b][j] node j's token (j >= 1)."""
    V = len(x)
    seen, count = np.zeros(V, bool), np.zeros(V)
    if history is not None:
        n = int(lens[b])
        n = n if 0 <= n <= history.shape[1] else 0
        p = min(max(int(prompt[b]), 0), n) if prompt is not None else 0
        for t, v in enumerate(history[b, :n]):
            if 0 <= v < V:
                seen[v] = True
                count[v] += t >= p
    if drafted is not None and is_tree(list(parent)):
        for j in path(parent, i)[1:]:
            v = int(drafted[b][j])
            if 0 <= v < V:
                seen[v] = True
                count[v] += 1
    y = np.array(x, np.float64)
    r = 1.0 if repetition is None else float(repetition[b])
    f = 0.0 if frequency is None else float(frequency[b])
    q = 0.0 if presence is None else float(presence[b])
    y = np.where(seen, np.where(y > 0, y / r, y * r), y)
    y = np.where(seen, y - (f * count + q * (count > 0)), y)
    if bias_ids is not None:
        for v, z in zip(bias_ids[b], bias_values[b]):
            if 0 <= v < V:
                y[v] += float(z)
    if allowed is not None:
        bits = (np.asarray(allowed[b, i]).astype(np.int64)[:, None] >> np.arange(32)) & 1
        y = np.where(bits.reshape(-1)[:V] != 0, y, -np.inf)
    return y


def keep(cache, path_nodes, accepted, lens, table):
    """cache [blocks, page, ...] as numpy, changed in place; the requests that are refused."""
    page, refused = cache.shape[1], []
    before = cache.copy()
    for b in range(len(accepted)):
        a, length = int(accepted[b]), int(lens[b])
        nodes = [int(p) for p in path_nodes[b][:max(a, -1) + 1]]
        room = table.shape[1] * page
        good = 0 <= a < path_nodes.shape[1] and length >= 0 and nodes[0] >= 0
        good = good and all(x < y for x, y in zip(nodes, nodes[1:])) and length + nodes[-1] < room
        places = [length + p for p in nodes] + [length + i for i in range(len(nodes))] if good else []
        if not good or any(not 0 <= table[b, t // page] < cache.shape[0] for t in places):
            refused.append(b)
            continue
        for i, p in enumerate(nodes):
            s, t = length + p, length + i
            cache[table[b, t // page], t % page] = before[table[b, s // page], s % page]
    return refused

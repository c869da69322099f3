"""Timed cases of the operators of a verification step between a model's
projections and its logits' use: new tokens into the paged cache (append_kv),
attention of drafted chains and trees over it (tree_attention), penalties,
biases and grammar masks on the logits (adjust_logits), and an accepted path's
cache entries moved together (keep_path).

run() computes a case in plain torch operations in 32 bits, or, where `own`
is true, through the library's calls.  exact() gives the same results from
the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
NEG_INF = float("-inf")


# ------------------------------------------------------------------ cases --


def _append(name, tokens, heads, kv_heads, dim, rot, dtype, page, last, norm=False, interleaved=False, skip=0.0):
    """last: the largest position; rot: how many of a head's dimensions turn;
    skip: share of tokens without a slot."""
    return dict(name=name, op="append", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot, dtype=dtype,
                page=page, last=last, norm=norm, interleaved=interleaved, skip=skip)


def _attend(name, B, nodes, form, heads, kv_heads, dim, length, dtype, page, by_head=False):
    """form: "chain", "tree" (one for the batch) or "dynamic" (a tree and a
    node count per request); length: the longest sequence (the shortest has a
    quarter of it); by_head: pages hold a head's entries together."""
    return dict(name=name, op="attend", B=B, nodes=nodes, form=form, heads=heads, kv_heads=kv_heads, dim=dim,
                length=length, dtype=dtype, page=page, by_head=by_head)


def _adjust(name, B, rows, V, dtype, history, form, bias, masked, penalised):
    """history: tokens of the longest request; form: "chain" or "tree"; bias:
    biased tokens per request; masked: share of requests under a grammar that
    allows one token in a hundred (-1: no masks at all); penalised: share of
    requests with penalties."""
    return dict(name=name, op="adjust", B=B, rows=rows, V=V, dtype=dtype, history=history, form=form, bias=bias,
                masked=masked, penalised=penalised)


def _keep(name, B, nodes, depth, planes, kv_heads, dim, dtype, page):
    """planes: key and value caches of all layers."""
    return dict(name=name, op="keep", B=B, nodes=nodes, depth=depth, planes=planes, kv_heads=kv_heads, dim=dim,
                dtype=dtype, page=page)


def listed():
    return [
        # a decoding step of 61 odd tokens: half-turned, interleaved heads with norms, some requests not served
        _append("append-decode-f16", 61, 24, 6, 96, 48, "f16", 48, 130000, norm=True, interleaved=True, skip=0.1),
        # prompts of several requests in one pass
        _append("append-prompt", 16384, 64, 8, 128, 128, "bf16", 64, 32768),
        # one request, 4 drafts after the last token, a small model: the latency of a layer
        _attend("attend-1req", 1, 5, "chain", 32, 8, 64, 1500, "bf16", 16),
        # 64 requests of 4 drafts at lengths of 2048 to 8192: bound by the cache's bytes
        _attend("attend-b64-chain", 64, 5, "chain", 64, 8, 128, 8192, "bf16", 16),
        # 32 requests of the 60-node tree: bound by the matrix products
        _attend("attend-b32-tree", 32, 60, "tree", 64, 8, 128, 8192, "bf16", 64),
        # trees per request, odd head size and page, grouped by five, fp16
        _attend("attend-dynamic-f16", 19, 45, "dynamic", 20, 4, 96, 3001, "f16", 48, by_head=True),
        # two long documents, single tokens: one row a head, split along the sequence
        _attend("attend-long", 2, 1, "chain", 64, 8, 128, 131072, "bf16", 128),
        # one request with 4 drafts, penalties, no grammar
        _adjust("adjust-1req", 1, 5, 128256, "bf16", 2000, "chain", 4, -1, 1.0),
        # the bench batch (256 requests, 8 drafts): a quarter under grammars, half with penalties
        _adjust("adjust-b256", 256, 9, 128256, "bf16", 4096, "chain", 16, 0.25, 0.5),
        # fp32 rows of an odd vocabulary over the 60-node tree, long histories, many biases
        _adjust("adjust-tree-odd-f32", 12, 60, 50021, "f32", 30000, "tree", 300, 0.5, 1.0),
        # one request's path, 16 layers
        _keep("keep-1req", 1, 16, 4, 32, 8, 64, "bf16", 16),
        # 32 requests of the 60-node tree, 40 layers
        _keep("keep-b32", 32, 60, 5, 80, 8, 128, "bf16", 16),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_ENTRIES = 2 * 131072 * 8  # cache entries (tokens times heads) of the largest listed calls
MOST_PRODUCTS = 32 * 60 * 64 * 5120 * 128  # multiplications of scores of the largest listed call


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "adjust", "adjust", "keep"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    page = rng.choice([8, 16, 32, 48, 64, 128])
    kv = rng.choice([1, 2, 4, 6, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    if op == "append":
        dim = rng.choice([64, 80, 96, 128])
        most = 16384 * 80 * 128 // ((group + 2) * kv * dim)
        c = _append("", _log_uniform(rng, 1, min(16384, most)), kv * group, kv, dim,
                    rng.choice([dim, dim, dim // 2]), dtype, page, _log_uniform(rng, 16, 1000000),
                    rng.random() < 0.5, rng.random() < 0.3, rng.choice([0.0, 0.2]))
    elif op == "attend":
        form = rng.choice(["chain", "chain", "tree", "dynamic"])
        nodes = _log_uniform(rng, 1, 17) if form == "chain" else _log_uniform(rng, 2, 100)
        B, dim = _log_uniform(rng, 1, 64), rng.choice([64, 64, 96, 128, 128])
        most = min(MOST_ENTRIES // (B * kv), MOST_PRODUCTS // (B * nodes * kv * group * dim), 131072)
        c = _attend("", B, nodes, form, kv * group, kv, dim, _log_uniform(rng, 1, max(2, most)), dtype, page,
                    rng.random() < 0.3)
    elif op == "adjust":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        V = _log_uniform(rng, 64, 262144)
        if rng.random() < 0.5:
            V = max(64, V // 64 * 64)
        form = rng.choice(["chain", "chain", "tree"])
        rows = rng.randint(1, 9) if form == "chain" else _log_uniform(rng, 2, 64)
        most = 256 * 9 * 128256 // (V * rows * (1 if dtype == "bf16" else 2))
        c = _adjust("", _log_uniform(rng, 1, max(1, min(256, most))), rows, V, dtype, _log_uniform(rng, 1, 30000), form,
                    rng.choice([0, 4, 300]), rng.choice([-1, 0.0, 0.5, 1.0]), rng.choice([0.0, 0.5, 1.0]))
    else:
        nodes = _log_uniform(rng, 2, 64)
        c = _keep("", _log_uniform(rng, 1, 32), nodes, rng.randint(1, min(8, nodes - 1)), 2 * rng.randint(1, 40), kv,
                  rng.choice([64, 96, 128]), dtype, page)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

_DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _some(n, share, g):
    """floor(n * share) random places of n, as a mask."""
    return torch.rand(n, generator=g, device=DEVICE).argsort() < int(n * share)


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device=DEVICE).to(dtype)


def _tree(n, depth, rng):
    """Parents of a random tree of n nodes in breadth-first order."""
    level, parent = [0], [-1]
    for i in range(1, n):
        low = max(parent[-1], 0)  # breadth first: parents do not go back
        high = min(i - 1, low + 3)
        p = int(rng.integers(low, high + 1))
        while level[p] >= depth:
            p -= 1
        p = max(p, parent[-1])
        if level[p] >= depth:
            p = parent[-1]
        parent.append(p)
        level.append(level[p] + 1)
    return parent


def _visible(parent):
    """[n, n]: node j is i or one of its ancestors."""
    n = len(parent)
    see = np.eye(n, dtype=bool)
    for i in range(1, n):
        see[i] |= see[parent[i]]
    return see


def _lengths(B, longest, g):
    """A quarter of the longest to the longest, evenly spread, in random order."""
    least = longest // 4
    lens = [longest if B == 1 else least + (longest - least) * i // (B - 1) for i in range(B)]
    order = torch.rand(B, generator=g, device=DEVICE).argsort()
    return torch.tensor(lens, dtype=torch.int32, device=DEVICE)[order]


def _table(need, spare, g):
    """Block tables of requests that need so many blocks, from a shuffled pool
    with some to spare; the entries behind are -1."""
    total, M = int(need.sum()) + spare, int(need.max())
    blocks = torch.randperm(total, generator=g, device=DEVICE).to(torch.int32)
    column = torch.arange(M, device=DEVICE)
    first = torch.cumsum(need, 0) - need
    place = (first[:, None] + column).clamp_(max=total - 1)
    return torch.where(column < need[:, None], blocks[place], -1).to(torch.int32), total


def _prepare_append(c, g):
    T, D, dt = c["tokens"], c["dim"], _DTYPE[c["dtype"]]
    H, K = c["heads"], c["kv_heads"]
    qkv = _normal((T, H + 2 * K, D), dt, g)  # the projection's output, all three in a row
    blocks = -(-T // c["page"]) + 2
    slots = torch.randperm(blocks * c["page"], generator=g, device=DEVICE)[:T].contiguous()
    slots[_some(T, c["skip"], g)] = -1
    positions = torch.randint(0, c["last"] + 1, (T,), generator=g, device=DEVICE).to(torch.int32)
    inv_freq = torch.tensor([500000.0 ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)], device=DEVICE)
    norm = dict(q_norm=_normal((D,), dt, g) * 0.2 + 1, k_norm=_normal((D,), dt, g) * 0.2 + 1) if c["norm"] else {}
    shape = (blocks, c["page"], K, D)
    return dict(case=c, q=qkv[:, :H], k=qkv[:, H:H + K], v=qkv[:, H + K:], slots=slots, positions=positions,
                inv_freq=inv_freq, norm=norm, k_cache=_normal(shape, dt, g), v_cache=_normal(shape, dt, g),
                out=dict(q=torch.empty(T, H, D, dtype=dt, device=DEVICE),
                         dev_error=torch.empty(1, dtype=torch.int32, device=DEVICE)))


def _prepare_attend(c, g, seed):
    B, N, D, K, dt = c["B"], c["nodes"], c["dim"], c["kv_heads"], _DTYPE[c["dtype"]]
    rng = np.random.default_rng(int(seed) * 104729 + 11)
    counts = np.full(B, N)
    if c["form"] == "dynamic":
        counts = np.array([N - (N // 2) * i // max(1, B - 1) for i in range(B)])[rng.permutation(B)]
    if c["form"] == "chain":
        parent, see = None, np.tril(np.ones((1, N, N), dtype=bool))
    elif c["form"] == "tree":
        tree = _tree(N, 6, rng)
        parent, see = np.array(tree), _visible(tree)[None]
    else:
        trees = [_tree(N, 6, rng) for _ in range(B)]
        parent, see = np.array(trees), np.stack([_visible(t) for t in trees])
    lens = _lengths(B, c["length"], g)
    n_nodes = torch.tensor(counts, dtype=torch.int32, device=DEVICE)
    table, blocks = _table((lens + N + c["page"] - 1) // c["page"], 1, g)
    # keys whose products with a query spread over a few units, as trained models' do
    shape = (blocks, K, c["page"], D) if c["by_head"] else (blocks, c["page"], K, D)
    k_cache, v_cache = _normal(shape, dt, g).mul_(1.5), _normal(shape, dt, g)
    if c["by_head"]:
        k_cache, v_cache = k_cache.transpose(1, 2), v_cache.transpose(1, 2)
    s = dict(case=c, q=_normal((B, N, c["heads"], D), dt, g), k_cache=k_cache, v_cache=v_cache, table=table, lens=lens,
             see=torch.tensor(see, device=DEVICE), n_nodes=n_nodes if c["form"] == "dynamic" else None,
             parent=None if parent is None else torch.tensor(parent, dtype=torch.int32, device=DEVICE),
             scale=1.0 / math.sqrt(D))
    # rows behind a request's nodes stay as they are
    s["out"] = dict(out=torch.zeros_like(s["q"]), dev_error=torch.empty(1, dtype=torch.int32, device=DEVICE))
    return s


def _prepare_adjust(c, g, seed):
    B, R, V = c["B"], c["rows"], c["V"]
    ints = dict(generator=g, device=DEVICE)
    logits = torch.randn(B, R, V, **ints).mul_(3.0).to(_DTYPE[c["dtype"]])
    L = c["history"]
    # text repeats itself: squares of uniform numbers favour low ids
    ids = (torch.rand(B, L, **ints).square() * V).to(torch.int32).clamp_(max=V - 1)
    lens = _lengths(B, L, g)
    prompt = (lens * torch.rand(B, **ints)).to(torch.int32)
    drafted = (torch.rand(B, R, **ints).square() * V).to(torch.int32).clamp_(max=V - 1)
    rng = np.random.default_rng(int(seed) * 104729 + 13)
    tree = _tree(R, 6, rng) if c["form"] == "tree" else list(range(-1, R - 1))
    see = _visible(tree)
    see[:, 0] = False  # the root's token is in the history
    free = ~_some(B, c["penalised"], g)
    repetition = (torch.rand(B, **ints) + 0.8).masked_fill_(free, 1.0)
    frequency = (torch.rand(B, **ints) - 0.2).masked_fill_(free, 0.0)
    presence = (torch.rand(B, **ints) - 0.2).masked_fill_(free, 0.0)
    s = dict(case=c, logits=logits, history=ids, history_lens=lens, prompt_lens=prompt, drafted=drafted,
             parent=torch.tensor(tree, dtype=torch.int32, device=DEVICE) if c["form"] == "tree" else None,
             see=torch.tensor(see, device=DEVICE), repetition=repetition, frequency=frequency, presence=presence,
             bias_ids=None, bias_values=None, allowed=None)
    if c["bias"]:
        s["bias_ids"] = torch.randint(0, V, (B, c["bias"]), **ints).to(torch.int32)
        s["bias_values"] = torch.randn(B, c["bias"], **ints).mul_(5.0)
    if c["masked"] >= 0:
        words = (V + 31) // 32
        allowed = torch.full((B, R, words), -1, dtype=torch.int32, device=DEVICE)
        ruled = _some(B, c["masked"], g)
        powers = 2 ** torch.arange(32, device=DEVICE)
        for b in ruled.nonzero()[:, 0].tolist():
            bits = torch.rand(R, words, 32, **ints) < 0.01
            bits[:, 0, 0] = True
            allowed[b] = (bits * powers).sum(2).to(torch.int32)
        s["allowed"] = allowed
    s["out"] = dict(logits=torch.empty_like(logits), dev_error=torch.empty(1, dtype=torch.int32, device=DEVICE))
    return s


def _prepare_keep(c, g, seed):
    B, N, P = c["B"], c["nodes"], c["page"]
    rng = np.random.default_rng(int(seed) * 104729 + 17)
    W = c["depth"] + 1
    path = np.full((B, W), -1)
    accepted = np.array([c["depth"] * (i + 1) // B for i in range(B)])[rng.permutation(B)]
    for b in range(B):
        a = int(accepted[b])
        # nodes behind those that are kept, so that a pass can be repeated on the same cache
        far = np.arange(a + 1, N)
        path[b, 0] = 0
        path[b, 1:a + 1] = np.sort(rng.permutation(far)[:a]) if len(far) >= a else np.arange(1, a + 1)
    lens = _lengths(B, 3 * P, g)
    table, blocks = _table((lens + N + P - 1) // P, 1, g)
    caches = _normal((c["planes"], blocks, P, c["kv_heads"], c["dim"]), _DTYPE[c["dtype"]], g)
    return dict(case=c, caches=caches, planes=list(caches.unbind(0)), lens=lens, table=table,
                path=torch.tensor(path, dtype=torch.int32, device=DEVICE),
                accepted=torch.tensor(accepted, dtype=torch.int32, device=DEVICE),
                out=dict(dev_error=torch.empty(1, dtype=torch.int32, device=DEVICE)))


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "append":
        return _prepare_append(case, g)
    if case["op"] == "attend":
        return _prepare_attend(case, g, seed)
    if case["op"] == "adjust":
        return _prepare_adjust(case, g, seed)
    return _prepare_keep(case, g, seed)


# ------------------------------------------------------------ plain forms --


def _turn(x, cos, sin, interleaved):
    """x [T, H, D] with its first 2 * cos.shape[1] dimensions turned."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=3).flatten(2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2)
    return torch.cat([turned, x[..., 2 * half:]], dim=2)


def _plain_append(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    q, k = s["q"].float(), s["k"].float()
    if c["norm"]:
        q = q * (q.square().mean(2, keepdim=True) + 1e-6).rsqrt() * s["norm"]["q_norm"].float()
        k = k * (k.square().mean(2, keepdim=True) + 1e-6).rsqrt() * s["norm"]["k_norm"].float()
    q = _turn(q, cos, sin, c["interleaved"]).to(s["q"].dtype)
    k = _turn(k, cos, sin, c["interleaved"]).to(s["q"].dtype)
    has = s["slots"] >= 0
    at = s["slots"][has]
    s["k_cache"].flatten(0, 1)[at] = k[has]
    s["v_cache"].flatten(0, 1)[at] = s["v"][has]
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_attend(s):
    c = s["case"]
    B, N, H, D = s["q"].shape
    K, P = c["kv_heads"], c["page"]
    table = s["table"].long().clamp(min=0)
    length = table.shape[1] * P
    keys = s["k_cache"][table].reshape(B, length, K, D).permute(0, 2, 1, 3).float()
    values = s["v_cache"][table].reshape(B, length, K, D).permute(0, 2, 1, 3).float()
    at = torch.arange(length, device=table.device)
    inside = at < (s["lens"][:, None] + N)  # [B, length]: entries that hold something
    values = torch.where(inside[:, None, :, None], values, 0.0)
    node = at - s["lens"][:, None]
    known = s["see"].expand(B, N, N).gather(2, node.clamp(0, N - 1)[:, None].expand(B, N, length))
    see = (node[:, None] < 0) | (known & (node[:, None] < N))
    if s["n_nodes"] is not None:
        see = see & (node < s["n_nodes"][:, None])[:, None]
    q = s["q"].float().view(B, N, K, H // K, D).permute(0, 2, 1, 3, 4).reshape(B, K, N * (H // K), D)
    scores = (q @ keys.transpose(2, 3)).mul_(s["scale"]).view(B, K, N, H // K, length)
    scores = torch.where(see[:, None, :, None], scores, NEG_INF)
    weights = (scores - scores.amax(4, keepdim=True).clamp(min=-1e30)).exp_()
    total = weights.sum(4, keepdim=True)
    out = (weights.view(B, K, N * (H // K), length) @ values).view(B, K, N, H // K, D) / total
    out = out.permute(0, 2, 1, 3, 4).reshape(B, N, H, D).to(s["q"].dtype)
    if s["n_nodes"] is not None:
        live = torch.arange(N, device=table.device) < s["n_nodes"][:, None]
        out = torch.where(live[:, :, None, None], out, s["out"]["out"])
    return out


def _allowed(words, V):
    bit = torch.arange(32, device=words.device)
    return ((words[..., None] >> bit) & 1).flatten(-2)[..., :V] != 0


def _plain_adjust(s):
    x = s["logits"].float()
    B, R, V = x.shape
    at = torch.arange(s["history"].shape[1], device=x.device)
    held = (at < s["history_lens"][:, None]).float()
    said = held * (at >= s["prompt_lens"][:, None])
    ids = s["history"].long()
    seen = torch.zeros(B, V, device=x.device).scatter_add_(1, ids, held)
    count = torch.zeros(B, V, device=x.device).scatter_add_(1, ids, said)
    path = torch.zeros(B, R, V, device=x.device)
    path.scatter_add_(2, s["drafted"].long()[:, None].expand(B, R, R), s["see"].float().expand(B, R, R))
    seen, count = seen[:, None] + path, count[:, None] + path
    each = (slice(None), None, None)
    r = s["repetition"][each]
    y = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    y = y - (s["frequency"][each] * count + s["presence"][each] * (count > 0))
    if s["bias_ids"] is not None:
        bias = torch.zeros(B, V, device=x.device).scatter_add_(1, s["bias_ids"].long(), s["bias_values"])
        y = y + bias[:, None]
    if s["allowed"] is not None:
        y = torch.where(_allowed(s["allowed"], V), y, NEG_INF)
    return y.to(s["logits"].dtype)


def _plain_keep(s):
    P = s["case"]["page"]
    W = s["path"].shape[1]
    i = torch.arange(W, device=s["path"].device)
    keep = i <= s["accepted"][:, None]

    def slot(place):
        return torch.gather(s["table"], 1, torch.div(place, P, rounding_mode="floor").long()).long() * P + place % P

    source = slot(s["lens"][:, None] + torch.where(keep, s["path"], i))[keep]
    target = slot(s["lens"][:, None] + i)[keep]
    flat = s["caches"].flatten(1, 2)
    flat[:, target] = flat[:, source]
    return s["caches"]


# ------------------------------------------------------------ library calls --


def _own_append(s):
    import speculative_decoding_verification_60_gb300 as sv

    out = sv.append_kv(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"], s["inv_freq"],
                       interleaved=s["case"]["interleaved"], out=s["out"], **s["norm"])
    return dict(q=out["q"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_attend(s):
    import speculative_decoding_verification_60_gb300 as sv

    return sv.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], parent=s["parent"],
                             n_nodes=s["n_nodes"], scale=s["scale"], out=s["out"])["out"]


def _own_adjust(s):
    import speculative_decoding_verification_60_gb300 as sv

    return sv.adjust_logits(s["logits"], history=s["history"], history_lens=s["history_lens"],
                            prompt_lens=s["prompt_lens"], drafted=s["drafted"], parent=s["parent"],
                            repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                            bias_ids=s["bias_ids"], bias_values=s["bias_values"], allowed=s["allowed"],
                            out=s["out"])["logits"]


def _own_keep(s):
    import speculative_decoding_verification_60_gb300 as sv

    sv.keep_path(s["planes"], s["path"], s["accepted"], s["lens"], s["table"], out=s["out"])
    return s["caches"]


def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _own_append(state) if own else _plain_append(state)
    if op == "attend":
        return _own_attend(state) if own else _plain_attend(state)
    if op == "adjust":
        return _own_adjust(state) if own else _plain_adjust(state)
    return _own_keep(state) if own else _plain_keep(state)


# ------------------------------------------------------------------- costs --


def work(case):
    c = case
    if c["op"] == "append":
        stored = c["tokens"] - int(c["tokens"] * c["skip"])
        values = c["tokens"] * c["heads"] + stored * 2 * c["kv_heads"]
        return dict(bytes=values * c["dim"] * 4 + 12 * c["tokens"], flops=4 * values * c["dim"])
    if c["op"] == "attend":
        N, B = c["nodes"], c["B"]
        tokens = B * (c["length"] + c["length"] // 4) // 2 if B > 1 else c["length"]
        nodes = B * N if c["form"] != "dynamic" else B * (N - N // 4)
        entries = tokens + nodes
        pairs = nodes * (tokens // B) + nodes * (N // 2 if c["form"] == "chain" else 4)
        return dict(bytes=entries * c["kv_heads"] * c["dim"] * 4 + nodes * c["heads"] * c["dim"] * 4,
                    flops=4 * pairs * c["heads"] * c["dim"])
    if c["op"] == "adjust":
        size = 2 if c["dtype"] == "bf16" else 4
        elements = c["B"] * c["rows"] * c["V"]
        ruled = int(c["B"] * max(c["masked"], 0.0)) * c["rows"] * c["V"]
        mask = elements // 8 if c["masked"] >= 0 else 0
        # a ruled-out token's logit is not read; requests without penalties need no history
        history = int(c["B"] * c["penalised"]) * c["history"] * 5 // 8 * 4
        return dict(bytes=(2 * elements - ruled) * size + mask + history + 8 * c["B"] * c["bias"], flops=2 * elements)
    accepted = [c["depth"] * (i + 1) // c["B"] for i in range(c["B"])]
    moved = sum(a for a in accepted if 2 * a < c["nodes"])  # as _prepare_keep makes them; a root stays
    return dict(bytes=max(1, moved) * c["planes"] * c["kv_heads"] * c["dim"] * 4, flops=0)


# ------------------------------------------------------------------- exact --


def _exact_append(s):
    c = s["case"]
    half = c["rot"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def one(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.square().mean(2, keepdim=True) + 1e-6).sqrt() * weight.double()
        x = x.clone()
        first = x[..., 0:2 * half:2] if c["interleaved"] else x[..., :half]
        second = x[..., 1:2 * half:2] if c["interleaved"] else x[..., half:2 * half]
        z = torch.complex(first.contiguous(), second.contiguous()) * turn
        first.copy_(z.real)
        second.copy_(z.imag)
        return x

    q, k = one(s["q"], s["norm"].get("q_norm")), one(s["k"], s["norm"].get("k_norm"))
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    live = (s["slots"] >= 0).nonzero()[:, 0]
    k_cache.flatten(0, 1)[s["slots"][live]] = k[live]
    v_cache.flatten(0, 1)[s["slots"][live]] = s["v"][live].double()
    return dict(q=q, k_cache=k_cache, v_cache=v_cache)


def _exact_attend(s):
    c = s["case"]
    B, N, H, D = s["q"].shape
    K, P = c["kv_heads"], c["page"]
    out = torch.zeros(B, N, H, D, dtype=torch.float64, device=DEVICE)
    for b, length in enumerate(s["lens"].tolist()):
        n = N if s["n_nodes"] is None else int(s["n_nodes"][b])
        place = torch.arange(length + n, device=DEVICE)
        block = s["table"][b, place // P].long()
        keys, values = s["k_cache"][block, place % P].double(), s["v_cache"][block, place % P].double()
        see = torch.ones(n, length + n, dtype=torch.bool, device=DEVICE)
        see[:, length:] = s["see"].expand(B, N, N)[b, :n, :n]
        for h in range(K):
            heads = slice(h * (H // K), (h + 1) * (H // K))
            q = s["q"][b, :n, heads].double()
            scores = torch.einsum("ngd,ld->ngl", q, keys[:, h]) * s["scale"]
            weights = torch.softmax(scores.masked_fill(~see[:, None], NEG_INF), 2)
            out[b, :n, heads] = torch.einsum("ngl,ld->ngd", weights, values[:, h])
    return out


def _exact_adjust(s):
    B, R, V = s["logits"].shape
    out = torch.empty(B, R, V, dtype=torch.float64, device=DEVICE)
    for b in range(B):
        n, p = int(s["history_lens"][b]), int(s["prompt_lens"][b])
        told = torch.bincount(s["history"][b, :n].long(), minlength=V)
        said = torch.bincount(s["history"][b, p:n].long(), minlength=V)
        for i in range(R):
            path = torch.bincount(s["drafted"][b][s["see"][i]].long(), minlength=V)
            x, count = s["logits"][b, i].double(), said + path
            r = s["repetition"][b].double()
            y = torch.where(told + path > 0, torch.where(x > 0, x / r, x * r), x)
            y = y - s["frequency"][b].double() * count - s["presence"][b].double() * (count > 0)
            if s["bias_ids"] is not None:
                y = y.index_add(0, s["bias_ids"][b].long(), s["bias_values"][b].double())
            if s["allowed"] is not None:
                y = y.masked_fill(~_allowed(s["allowed"][b, i], V), NEG_INF)
            out[b, i] = y
    return out


def exact(case, seed):
    if case["op"] == "keep":
        return None  # entries are moved, not computed
    state = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "adjust": _exact_adjust}[case["op"]](state)
